// One token per row of logits, from a given uniform random number.
//
// With m the row's largest logit and t its temperature, token i weighs w_i = exp((x_i - m)/t).
// The kept tokens are a prefix of the order "larger logit first, lower index first among
// equals": the shortest of the prefixes that top-k, top-p (mass before the token below
// top_p times the mass of the top-k survivors) and min-p (w_i >= min_p) allow.  The sampled
// token is the first in vocabulary order whose cumulated kept weight exceeds u times the total.
// t = 0 keeps the largest logit alone.
//
// Weights (to 2e-13 of themselves) and the sums that decide a token are in 64 bits: a token is
// decided by where u * total falls between two of up to a million borders, and 32-bit weights (1e-7
// each) would put one draw in some thousands on the wrong side.  The exponential is the cost (ten 64-bit
// operations, half rate), so each row takes the way with the fewest of them:
//   t = 0          the largest logit: one read of the row, no weight.
//   small top-k    every thread keeps the largest logit of its stripe.  The k-th largest of
//                  these 512 or 1024 is at most the k-th largest logit, so the few logits above it hold
//                  the prefix; only threads whose own maximum reaches it read their stripe
//                  again.  What is left is a list of k to a few k tokens in shared memory.
//   top-p          a second read sums all weights and counts tokens into 2048 bins of the
//                  weight's logarithm, whose masses are known well enough (1e-4) to name the
//                  bin of the border; a third read sums what lies above it by segments of the
//                  vocabulary and lists the border's bins, where the border is found exactly.
//                  Bins that hold more than the list are counted once more into 2048 parts of
//                  their range of logits (for 16-bit logits, or such widened to 32: one part
//                  per value, and the border is known), and a fourth read does the rest.
//   otherwise      a second read sums the kept weights by segments.
//   bf16 logits    (top-p and otherwise) take few values: those of a magnitude from 2^-8 to 2^8 have
//                  a counter and a weight each in shared memory, so a weight is computed once for
//                  a value (4096 of them) and not for a logit, top-p's border is known from the
//                  counts alone, and the sums by segments look weights up.  The few others go by
//                  the exponential.
// 2048 rows of 65536 bf16 logits with mixed filters take 205 us (268 MB; greedy alone 59 us, 4.6 TB/s;
// top-k of 50 114 us, no filter 208 us, top-p 308 us), 128 rows of 100003 in fp32 105 us, one of 32768
// with top-p 25 to 50 us by temperature and top_p: instructions and the barriers between a row's steps bound it, not bytes.
// The segment that holds the token is then read once more.  Where a list overflows or top-k is
// large, the border comes from a radix descent over the logits' bits, general and slow: its atomics
// meet in a few of 256 counters (top-k of 1000: 1.2 ms for one row of 32768, 3.6 ms for the 128 rows,
// 19 ms for the 2048; with top-p 7% more).
// Second and later reads hit L2.
#include <math_constants.h>

#include "serving.cuh"

namespace tv {
namespace {

constexpr int kMaxWarps = 32;                  // of a row's CTA: 512 or 1024 threads
constexpr int kList = 1024;                    // candidates held in shared memory
constexpr int kSmallK = 256;                   // largest top-k that goes by stripe maxima
constexpr int kBins = 2048;
constexpr float kOctaves = 48.f;               // the bins' range: weights down to 2^-48
constexpr float kPhase = 2048.f;               // steps of a token's place in its bin: a million fit 32 bits
constexpr double kScale = 4398046511104.0;     // 2^42: a million weights stay below 2^62, twice over
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // key of -inf
constexpr unsigned kFull = 0xffffffffu;

using u64 = unsigned long long;

// Monotone key: larger float, larger key.  -0 counts as +0 (NaN is made -inf on loading).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// A listed token: larger logit first, lower index first.
__device__ __forceinline__ u64 entry_of(uint32_t key, int i) {
  return (u64)key << 32 | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ uint32_t entry_key(u64 e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ int entry_index(u64 e) { return (int)(0xFFFFFFFFu - (uint32_t)e); }

struct SampleSmem {
  double table[16];                            // 2^(j/16)
  union {
    struct { unsigned count[kBins], phase[kBins]; } bin;
    struct { u64 sum[256], low[256]; } hist;
    struct { double w[kList], w_by_index[kList]; } list_w;
  };
  u64 list[kList], sorted[kList];
  double part[kMaxWarps];
  int ipart[kMaxWarps];
  int n, pick, ties_left, equals, around[2];
  uint32_t digit;
  u64 before[2];                               // a Mass
  double goal;
};

// A sum of weights (of at most 1) as two integers, in steps of 2^-42 and of 2^-84, whose order in the atomics
// does not matter.  The second holds what the first leaves: the border of a top_p next to 1 lies among
// weights of 2^-43, and a sum over a million tokens has to be known to a small part of one.
struct Mass {
  u64 sum, low;
  static __device__ __forceinline__ Mass of(double w) {
    const double x = w * kScale, whole = floor(x);
    return {(u64)whole, (u64)__double2ll_rn((x - whole) * kScale)};
  }
  __device__ __forceinline__ void add(Mass o) { sum += o.sum; low += o.low; }
  __device__ __forceinline__ double value() const { return (double)sum + (double)low / kScale; }   // times 2^42
};

// exp((x - m) / t) in 64 bits, as 2^(i/16 + r): a table of 2^(j/16), whose 16 entries lie in
// banks of their own, and five terms of the exponential series in r (|r ln 2| < 0.022: 1.4e-13
// relative).  Adding 1.5 * 2^48 rounds to sixteenths and leaves i in the low word.  What weighs
// less than 2^-1000 weighs nothing.
struct Weigher {
  float max;
  double m, c;                                 // c = log2(e) / t
  const double *table;
  __device__ __forceinline__ double operator()(float x) const {
    if (max == CUDART_INF_F) return x == max ? 1.0 : 0.0;
    constexpr double kMagic = 422212465065984.0;
    const double d = (double)x - m, s = fma(d, c, kMagic), r = fma(d, c, kMagic - s);
    const int i = __double2loint(s), above = __double2hiint(s) - 0x42F80000;
    double p = fma(r, 1.3333558146428443e-3, 9.6181291076284772e-3);
    p = fma(p, r, 5.5504108664821580e-2);
    p = fma(p, r, 2.4022650695910072e-1);
    p = fma(p, r, 6.9314718055994531e-1);
    const double y = table[i & 15], w = fma(y, p * r, y);
    const bool in = above == i >> 31 && i >= -16000;          // -1000 <= z <= 0 (-inf is not)
    return in ? __hiloint2double(__double2hiint(w) + ((i >> 4) << 20), __double2loint(w)) : 0.0;
  }
};

// Values of bf16 logits with a place of their own: magnitudes from 2^-8 up to 2^8, 128 to an octave.
constexpr int kValues = 4096;
struct ValueSmem {
  double w[kValues];
  unsigned count[kValues];
};
constexpr uint32_t kFirstMagnitude = 0x3B80u;  // 2^-8
// Place of the logit with these 16 bits: its magnitude's, and 2048 more for negative ones; at least
// kValues for those without one.
__device__ __forceinline__ uint32_t place_of(uint32_t bits) {
  const uint32_t n = (bits & 0x7FFFu) - kFirstMagnitude;
  return n < 2048u ? n | (bits & 0x8000u) >> 4 : kValues;
}
__device__ __forceinline__ float value_at(int place) {
  return __uint_as_float((kFirstMagnitude + (place & 2047)) << 16 | (uint32_t)(place & 2048) << 20);
}

// A row of logits by aligned 16-byte vectors; the first and the last may be partial.
template <typename T> struct Row {
  static constexpr int N = 16 / sizeof(T);
  const T *x;
  int V, off;                                  // off: elements of vector 0 before the row
  int vectors, full0, full1;                   // all, and the range that is whole
  __device__ __forceinline__ Row(const T *p, int n) : x(p), V(n) {
    off = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    vectors = (off + V + N - 1) / N;
    full0 = off ? 1 : 0;
    full1 = max(full0, (off + V) / N);
  }
  static __device__ __forceinline__ void widen(uint4 r, float (&v)[N]);
  __device__ __forceinline__ uint4 raw(int vi) const {
    return *reinterpret_cast<const uint4 *>(x - off + (long long)vi * N);
  }
  __device__ __forceinline__ int index(int vi, int j) const { return vi * N + j - off; }
  // Vector vi, -inf in the places outside the row and for NaN.
  __device__ __forceinline__ void load(int vi, float (&v)[N]) const {
    if (vi >= full0 && vi < full1) {
      widen(raw(vi), v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = fmaxf(v[j], -CUDART_INF_F);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = index(vi, j);
        v[j] = i >= 0 && i < V ? fmaxf(to_f32(x[i]), -CUDART_INF_F) : -CUDART_INF_F;
      }
    }
  }
};
template <> __device__ __forceinline__ void Row<float>::widen(uint4 r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
  v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
}
template <> __device__ __forceinline__ void Row<__nv_bfloat16>::widen(uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Inclusive prefix over the warp.
template <typename U> __device__ __forceinline__ U warp_scan(U v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const U y = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Sums over the block in a fixed order; every thread gets the result.  (Each warp goes through the
// warps' parts by shuffles: five steps where adding them up in a row takes 32.)
template <int kThreads>
__device__ __forceinline__ double block_sum(double v, double *part) {
  constexpr int kWarps = kThreads / 32;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < kWarps ? part[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Exclusive prefix over the block's threads of a sum and a count.
template <int kThreads>
__device__ __forceinline__ void block_scan(double v, int c, SampleSmem &sm, double &v_before,
                                           int &c_before, double &v_all, int &c_all) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const double s = warp_scan(v);
  const int k = warp_scan(c);
  __syncthreads();
  if (lane == 31) {
    sm.part[warp] = s;
    sm.ipart[warp] = k;
  }
  __syncthreads();
  const double parts = warp_scan(lane < kWarps ? sm.part[lane] : 0.0);
  const int iparts = warp_scan(lane < kWarps ? sm.ipart[lane] : 0);
  v_all = __shfl_sync(kFull, parts, 31);
  c_all = __shfl_sync(kFull, iparts, 31);
  const double b = __shfl_sync(kFull, parts, max(warp - 1, 0)), up = __shfl_up_sync(kFull, s, 1);
  const int kb = __shfl_sync(kFull, iparts, max(warp - 1, 0));
  v_before = (warp ? b : 0.0) + (lane ? up : 0.0);
  c_before = (warp ? kb : 0) + k - c;
}

// sorted = list[0..n) in falling order, by counting what is larger (the entries differ).
template <int kThreads>
__device__ __forceinline__ void sort_list(const u64 *list, u64 *sorted, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 e = list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > e;
    sorted[rank] = e;
  }
}

__device__ __forceinline__ void put_token(const SampleArgs &a, int row, int token, double p) {
  a.token[row] = token;
  if (a.logprob) a.logprob[row] = (float)log(p);
}

// The token among the first n listed ones (sm.sorted, all kept, weights in sm.list_w.w): by index
// order.  Called by the whole block.
template <int kThreads>
__device__ void pick_from_list(const SampleArgs &a, int row, SampleSmem &sm, int n, double u) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t idx = (uint32_t)sm.sorted[i];           // falls as the index rises
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += (uint32_t)sm.sorted[j] > idx;
    sm.list[rank] = sm.sorted[i];
    sm.list_w.w_by_index[rank] = sm.list_w.w[i];
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x, per = (n + 31) / 32, lo = min(n, lane * per), hi = min(n, lo + per);
  double own = 0.0;
  for (int i = lo; i < hi; ++i) own += sm.list_w.w_by_index[i];
  double s = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += y;
  }
  const double total = __shfl_sync(kFull, s, 31), target = u * total;
  const unsigned live = __ballot_sync(kFull, own > 0.0);
  const unsigned hit = __ballot_sync(kFull, own > 0.0 && s > target);
  const int src = hit ? __ffs(hit) - 1 : 31 - __clz(live);
  double c = __shfl_up_sync(kFull, s, 1);
  if (lane == 0) c = 0.0;
  if (lane == src) {
    int at = lo;
    for (int i = lo; i < hi; ++i) {
      const double w = sm.list_w.w_by_index[i];
      if (w > 0.0) at = i;
      c += w;
      if (w > 0.0 && c > target) break;
    }
    put_token(a, row, entry_index(sm.list[at]), sm.list_w.w_by_index[at] / total);
  }
}

// Sorts the listed tokens and weighs them (sm.sorted, sm.list_w.w); returns how many of them start
// below top_p of the mass, `above` of which lies before the list and `below` behind it, or 0 if
// the border is not inside it.  Called by the whole block.
template <int kThreads>
__device__ int border_in_list(const Weigher &weight, SampleSmem &sm, int n, double above, double below,
                              double top_p) {
  sort_list<kThreads>(sm.list, sm.sorted, n);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    sm.list_w.w[i] = weight(value_of(entry_key(sm.sorted[i])));
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (n + 31) / 32, lo = min(n, lane * per), hi = min(n, lo + per);
    double s = 0.0;
    for (int i = lo; i < hi; ++i) s += sm.list_w.w[i];
    const double mine = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    const double end = above + __shfl_sync(kFull, s, 31), goal = top_p * (end + below);
    double at = above + (s - mine);
    int kept = 0;
    for (int i = lo; i < hi; ++i) {
      kept += at < goal;
      at += sm.list_w.w[i];
    }
    kept = __reduce_add_sync(kFull, kept);
    // inside: the first listed token is kept, and the list ends at or past the goal
    if (lane == 0) sm.pick = kept > 0 && (kept < n || end >= goal) ? kept : 0;
  }
  __syncthreads();
  return sm.pick;
}

// The nearest bins with tokens on either side of sm.pick (itself where there is none; the last
// bin, of the weights below the range, does not count).  Called by the whole block.
template <int kThreads>
__device__ void filled_around(SampleSmem &sm, int &before, int &after) {
  __syncthreads();
  const int pick = sm.pick;
  int lo = -1, hi = kBins;
#pragma unroll
  for (int j = 0; j < kBins / kThreads; ++j) {
    const int b = threadIdx.x * (kBins / kThreads) + j;
    if (sm.bin.count[b] && b < kBins - 1) {
      if (b < pick) lo = max(lo, b);
      if (b > pick) hi = min(hi, b);
    }
  }
  lo = __reduce_max_sync(kFull, lo);
  hi = __reduce_min_sync(kFull, hi);
  if (threadIdx.x == 0) {
    sm.around[0] = -1;
    sm.around[1] = kBins;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&sm.around[0], lo);
    atomicMin(&sm.around[1], hi);
  }
  __syncthreads();
  before = sm.around[0] < 0 ? pick : sm.around[0];
  after = sm.around[1] == kBins ? pick : sm.around[1];
}

// Border of top-k (by count) or of top-p (by mass) through the bits of the keys, eight at a time.
// General and slow: four reads of the row.  sm.equals is the number of logits at top-k's border.
template <int kThreads, typename T>
__device__ void descend(const Row<T> &row, const Weigher &weight, SampleSmem &sm, bool by_mass,
                        int top_k, float top_p, uint32_t &edge, int &n_edge) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (tid < 256) sm.hist.sum[tid] = sm.hist.low[tid] = 0;
    if (tid < 2 && shift == 24) sm.before[tid] = 0;      // (a descent before this one has been read)
    __syncthreads();
    for (int i = tid; i < row.V; i += kThreads) {
      const float x = fmaxf(to_f32(row.x[i]), -CUDART_INF_F);
      const uint32_t key = key_of(x);
      if (key >= edge && (key & mask) == prefix) {
        const Mass m = by_mass ? Mass::of(weight(x)) : Mass{1, 0};
        atomicAdd(&sm.hist.sum[key >> shift & 255], m.sum);
        if (m.low) atomicAdd(&sm.hist.low[key >> shift & 255], m.low);
      }
    }
    __syncthreads();
    if (tid == 0) {
      if (shift == 24) {
        // the first read has all the mass; of the equals at top-k's border only n_edge count
        Mass all = {0, 0};
        for (int d = 0; d < 256; ++d) all.add({sm.hist.sum[d], sm.hist.low[d]});
        const Mass e = Mass::of(edge ? weight(value_of(edge)) : 0.0);
        const u64 out = edge ? sm.equals - n_edge : 0;
        sm.goal = by_mass ? (double)top_p * Mass{all.sum - out * e.sum, all.low - out * e.low}.value()
                          : (double)top_k;
      }
      Mass c = {sm.before[0], sm.before[1]}, at = c;
      int pick = -1;
      for (int d = 255; d >= 0; --d) {
        const Mass m = {sm.hist.sum[d], sm.hist.low[d]};
        if (!(m.sum || m.low)) continue;
        // the last digit that starts below the goal (the first one always does or is taken)
        if (pick >= 0 && !(c.value() < sm.goal)) break;
        pick = d;
        at = c;
        c.add(m);
      }
      sm.digit = pick;
      sm.before[0] = at.sum;
      sm.before[1] = at.low;
      if (!by_mass) sm.equals = (int)(c.sum - at.sum);
    }
    __syncthreads();
    prefix |= sm.digit << shift;
    mask |= 255u << shift;
  }
  if (!by_mass) {
    edge = prefix;
    n_edge = top_k - (int)sm.before[0];
    return;
  }
  // equals at the border: kept while the mass before them is below the goal
  const double w = weight(value_of(prefix)) * kScale;
  const int most = prefix == edge ? n_edge : row.V;
  int n = 1;
  if (w > 0.0) {
    const double d = (sm.goal - Mass{sm.before[0], sm.before[1]}.value()) / w;
    n = d >= (double)most ? most : max(1, (int)ceil(d));
  }
  edge = prefix;
  n_edge = min(n, most);
}

// bf16 logits: the border of top-p and the kept weight above it in this warp's segment of vectors
// [s0, s1), with the border's equals there, by values.  False (nothing is known) where logits without
// a place weigh too much for it.  Called by the whole block.
template <int kThreads>
__device__ bool by_values(const Row<__nv_bfloat16> &row, const Weigher &weight, SampleSmem &sm, ValueSmem &vs,
                          float t, float top_p, float min_p, bool border, uint32_t &edge, int &n_edge, int s0,
                          int s1, double &kept, int &ties) {
  const int tid = threadIdx.x, lane = tid & 31;
  const float top = weight.max;
  // what lies below weighs less than 2^-1000
  const float nothing = fmaxf(__double2float_rd((double)top - 700.0 * (double)t), -3.4028234e38f);
  constexpr int kPer = kValues / kThreads;
  // places in falling order of their values: positive ones from the largest on, then negative ones
  const auto place_in_order = [](int p) { return p < 2048 ? 2047 - p : p; };
  double mass[kPer], mine = 0.0;
  if (border) {
    for (int i = tid; i < kValues; i += kThreads) vs.count[i] = 0;
    if (tid == 0) {
      sm.n = 0;
      sm.pick = -1;
    }
    __syncthreads();
    for (int vi = tid; vi < row.vectors; vi += kThreads) {
      if (vi >= row.full0 && vi < row.full1) {
        const uint4 r = row.raw(vi);
        const uint32_t word[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t bits = j & 1 ? word[j / 2] >> 16 : word[j / 2] & 0xFFFFu, p = place_of(bits);
          if (p < kValues) {
            atomicAdd(&vs.count[p], 1u);
          } else if (fmaxf(__uint_as_float(bits << 16), -CUDART_INF_F) >= nothing) {
            const int at = atomicAdd(&sm.n, 1);
            if (at < kList) sm.list[at] = entry_of(key_of(__uint_as_float(bits << 16)), row.index(vi, j));
          }
        }
      } else {
        for (int j = 0; j < 8; ++j) {
          const int i = row.index(vi, j);
          if (i < 0 || i >= row.V) continue;
          const float x = fmaxf(to_f32(row.x[i]), -CUDART_INF_F);
          const uint32_t p = place_of(__float_as_uint(x) >> 16);
          if (p < kValues) {
            atomicAdd(&vs.count[p], 1u);
          } else if (x >= nothing) {
            const int at = atomicAdd(&sm.n, 1);
            if (at < kList) sm.list[at] = entry_of(key_of(x), i);
          }
        }
      }
    }
    __syncthreads();
    if (sm.n > kList) return false;
    // the listed ones: small magnitudes, all between the positive and the negative places
    double small = 0.0;
    bool large = false;
    for (int i = tid; i < sm.n; i += kThreads) large |= fabsf(value_of(entry_key(sm.list[i]))) > 1.f;
    if (__syncthreads_or(large)) return false;
    // (summed by falling entries, so that the order of the list does not matter)
    sort_list<kThreads>(sm.list, sm.sorted, sm.n);
    __syncthreads();
    for (int i = tid; i < sm.n; i += kThreads) small += weight(value_of(entry_key(sm.sorted[i])));
    small = block_sum<kThreads>(small, sm.part);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int p = place_in_order(tid * kPer + j);
      const unsigned n = vs.count[p];
      const double w = n ? weight(value_at(p)) : 0.0;
      vs.w[p] = w;
      mass[j] = n * w;
      mine += mass[j];
    }
    double c, all;
    int unused, unused_all;
    block_scan<kThreads>(mine, 0, sm, c, unused, all, unused_all);
    all += small;
    if (tid * kPer >= 2048) c += small;
    const double goal = (double)top_p * all;
    // the last value that starts below the goal
    int last = -1;
    double start = 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (mass[j] > 0.0 && c < goal) {
        last = tid * kPer + j;
        start = c;
      }
      c += mass[j];
    }
    const int warp_last = __reduce_max_sync(kFull, last);
    if (lane == 0) atomicMax(&sm.pick, warp_last);
    __syncthreads();
    const int pick = sm.pick;
    if (pick >= 0 && pick == last) {
      const int p = place_in_order(pick), n = (int)vs.count[p];
      const double d = (goal - start) / vs.w[p];
      // (0: the goal lies behind this value's equals, among the small magnitudes)
      sm.ties_left = d <= (double)n ? max(1, (int)ceil(d)) : sm.n == 0 ? n : 0;
    }
    __syncthreads();
    if (pick < 0 || sm.ties_left == 0) return false;
    edge = key_of(value_at(place_in_order(pick)));
    n_edge = sm.ties_left;
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int p = place_in_order(tid * kPer + j);
      const float x = value_at(p);
      vs.w[p] = x <= top ? weight(x) : 0.0;
    }
  }
  // what is kept: values above the border and heavy enough; its equals are counted apart
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int p = place_in_order(tid * kPer + j);
    if (key_of(value_at(p)) <= edge || vs.w[p] < (double)min_p) vs.w[p] = 0.0;
  }
  const uint32_t edge_place = edge ? place_of(__float_as_uint(value_of(edge)) >> 16) : kValues + 1;
  __syncthreads();
  kept = 0.0;
  ties = 0;
  for (int vi = s0 + lane; vi < s1; vi += 32) {
    if (vi >= row.full0 && vi < row.full1) {
      const uint4 r = row.raw(vi);
      const uint32_t word[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t bits = j & 1 ? word[j / 2] >> 16 : word[j / 2] & 0xFFFFu, p = place_of(bits);
        if (p < kValues) {
          kept += vs.w[p];
          ties += p == edge_place;
        } else {
          const float x = fmaxf(__uint_as_float(bits << 16), -CUDART_INF_F);
          if (x >= nothing && key_of(x) > edge) {
            const double w = weight(x);
            if (w >= (double)min_p) kept += w;
          } else if (edge_place == kValues) {
            ties += key_of(x) == edge;
          }
        }
      }
    } else {
      float v[8];
      row.load(vi, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t key = key_of(v[j]);
        if (key > edge) {
          const double w = weight(v[j]);
          if (w >= (double)min_p) kept += w;
        } else {
          ties += key == edge;
        }
      }
    }
  }
  return true;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(SampleArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int N = Row<T>::N;
  constexpr bool kByValues = sizeof(T) == 2;
  __shared__ SampleSmem sm;
  extern __shared__ __align__(16) unsigned char smem_dyn[];
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<T> row(static_cast<const T *>(a.logits) + (long long)r * a.stride, a.V);
  const float u = a.uniform[r], t = a.temperature ? a.temperature[r] : 1.f;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
  const int k_asked = a.top_k ? a.top_k[r] : 0, top_k = k_asked > 0 && k_asked < a.V ? k_asked : 0;
  if (!(u >= 0.f && u <= 1.f && t >= 0.f && t < CUDART_INF_F && top_p >= 0.f && top_p <= 1.f &&
        min_p >= 0.f && min_p <= 1.f)) {
    if (tid == 0) set_status(a.ws, TV_ERR_BAD_PARAM, r);
    return;
  }

  // ---- first read: the largest logit of each thread's stripe, and of the row ---------------
  float own = -CUDART_INF_F;
#pragma unroll 4
  for (int vi = row.full0 + tid; vi < row.full1; vi += kThreads) {
    float v[N];
    Row<T>::widen(row.raw(vi), v);
#pragma unroll
    for (int j = 0; j < N; ++j) own = fmaxf(own, v[j]);      // a NaN loses
  }
  // the partial vectors belong to the last two threads' stripes
  const int ragged = tid == kThreads - 1 && row.full0 > 0 ? 0
                     : tid == kThreads - 2 && row.full1 < row.vectors ? row.full1 : -1;
  if (ragged >= 0) {
    float v[N];
    row.load(ragged, v);
#pragma unroll
    for (int j = 0; j < N; ++j) own = fmaxf(own, v[j]);
  }
  const uint32_t own_key = key_of(own);
  uint32_t max_key = __reduce_max_sync(kFull, own_key);
  if (lane == 0) sm.ipart[warp] = (int)max_key;
  if (tid < 16) sm.table[tid] = exp2((double)tid / 16.0);
  if (tid == 0) sm.n = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) max_key = max(max_key, (uint32_t)sm.ipart[w]);
  if (max_key == kKeyNegInf) {
    if (tid == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -CUDART_INF_F;
    }
    return;
  }
  const float top = value_of(max_key);
  // visits the stripe of this thread again: f(value, index)
  const auto stripe = [&](auto f) {
#pragma unroll 4
    for (int vi = row.full0 + tid; vi < row.full1; vi += kThreads) {
      float v[N];
      Row<T>::widen(row.raw(vi), v);
#pragma unroll
      for (int j = 0; j < N; ++j) f(fmaxf(v[j], -CUDART_INF_F), row.index(vi, j));
    }
    if (ragged >= 0) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = row.index(ragged, j);
        if (i >= 0 && i < row.V) f(fmaxf(to_f32(row.x[i]), -CUDART_INF_F), i);
      }
    }
  };

  // ---- temperature zero, or one token kept: the lowest index of the largest logit ---------
  if (t == 0.f || top_k == 1 || top_p == 0.f) {
    unsigned first = 0xFFFFFFFFu;
    if (own_key == max_key)
      stripe([&](float x, int i) { if (x == top) first = min(first, (unsigned)i); });
    first = __reduce_min_sync(kFull, first);
    __syncthreads();
    if (lane == 0) sm.ipart[warp] = (int)first;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) first = min(first, (unsigned)sm.ipart[w]);
      a.token[r] = (int)first;
      if (a.logprob) a.logprob[r] = 0.f;
    }
    return;
  }

  const Weigher weight{top, (double)top, 1.4426950408889634 / (double)t, sm.table};
  uint32_t edge = 0;                  // kept: keys above `edge`, and the first n_edge equal to it
  int n_edge = a.V;
  bool by_edge = false;               // the border is known from a descent

  // ---- small top-k: a short list ------------------------------------------------------------
  if (top_k && top_k <= kSmallK) {
    // a bound that at least top_k logits reach: the top_k-th largest stripe maximum, to 20 bits
    uint32_t bound = 0;
    for (uint32_t bit = 1u << 31; bit >= 1u << 12; bit >>= 1)
      if (__syncthreads_count(own_key >= (bound | bit)) >= top_k) bound |= bit;
    // exp(-760) is zero in 64 bits: logits below that (masked ones) are not worth a place
    const float bound_x = fmaxf(value_of(max(bound, kKeyNegInf)), top - 760.f * t);
    if (own_key >= bound)
      stripe([&](float x, int i) {
        if (x >= bound_x && x > -CUDART_INF_F) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < kList) sm.list[at] = entry_of(key_of(x), i);
        }
      });
    __syncthreads();
    const int n = sm.n, k = min(top_k, n);
    if (n <= kList) {
      sort_list<kThreads>(sm.list, sm.sorted, n);
      __syncthreads();
      for (int i = tid; i < k; i += kThreads)
        sm.list_w.w[i] = weight(value_of(entry_key(sm.sorted[i])));
      __syncthreads();
      if (warp == 0) {
        // the prefixes of top-p and min-p: lanes take runs of the sorted list
        const int per = (k + 31) / 32, lo = min(k, lane * per), hi = min(k, lo + per);
        double s = 0.0;
        for (int i = lo; i < hi; ++i) s += sm.list_w.w[i];
        const double mine = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(kFull, s, o);
          if (lane >= o) s += y;
        }
        const double goal = (double)top_p * __shfl_sync(kFull, s, 31);
        double c = s - mine;
        int kept = 0;
        for (int i = lo; i < hi; ++i) {
          const double w = sm.list_w.w[i];
          kept += (i == 0 || top_p >= 1.f || c < goal) && w >= (double)min_p;
          c += w;
        }
        kept = __reduce_add_sync(kFull, kept);
        if (lane == 0) sm.pick = kept;
      }
      __syncthreads();
      pick_from_list<kThreads>(a, r, sm, sm.pick, (double)u);
      return;
    }
    __syncthreads();
  }
  if (top_k) {
    descend<kThreads>(row, weight, sm, false, top_k, top_p, edge, n_edge);
    by_edge = true;
  }

  // ---- top-p: the border ---------------------------------------------------------------------
  const int seg = (row.vectors + kWarps - 1) / kWarps;        // vectors per warp's segment
  const int s0 = min(row.vectors, warp * seg), s1 = min(row.vectors, s0 + seg);
  double kept_here = 0.0;             // kept weight above the border in this warp's segment
  int ties = 0;                       // equals of the border in it
  bool have_sums = false;
  if constexpr (kByValues) {
    if (by_edge && top_p < 1.f) descend<kThreads>(row, weight, sm, true, top_k, top_p, edge, n_edge);
    __syncthreads();
    if (top < CUDART_INF_F)
      have_sums = by_values<kThreads>(row, weight, sm, *reinterpret_cast<ValueSmem *>(smem_dyn), t, top_p, min_p,
                            top_p < 1.f && !by_edge, edge, n_edge, s0, s1, kept_here, ties);
    __syncthreads();
    if (!have_sums && tid == 0) sm.n = 0;
    __syncthreads();
  }
  if (have_sums) {
  } else if (top_p < 1.f && !by_edge) {
    int listed = 0;                   // tokens of the list before the border
    const float scale = (float)(weight.c * (double)(kBins / kOctaves));
    const auto bin_of = [&](float x, float &z) {
      z = (top - x) * scale;
      if (x == top) z = 0.f;
      return min((int)z, kBins - 1);                          // monotone in x; saturates
    };
    for (int i = tid; i < kBins; i += kThreads) sm.bin.count[i] = sm.bin.phase[i] = 0;
    __syncthreads();
    unsigned bits = 0;                // that any logit has
    stripe([&](float x, int) {
      float z;
      bits |= __float_as_uint(x);
      const int b = bin_of(x, z);
      if (b < kBins - 1) {
        atomicAdd(&sm.bin.count[b], 1u);
        atomicAdd(&sm.bin.phase[b], (unsigned)((z - (float)b) * kPhase));
      }
    });
    __syncthreads();
    // approximate masses: a bin's tokens at their mean place in it (1e-5: the bin is 1.6% wide)
    constexpr int kPer = kBins / kThreads;
    double mass[kPer], mine = 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int b = tid * kPer + j;
      const float count = (float)sm.bin.count[b];
      const float place = ((float)sm.bin.phase[b] / fmaxf(count, 1.f) + 0.5f) / kPhase;
      mass[j] = (double)count * exp2f(-((float)b + place) * (kOctaves / kBins));
      mine += mass[j];
    }
    double c, all;
    int unused, unused_all;
    block_scan<kThreads>(mine, 0, sm, c, unused, all, unused_all);
    double goal = (double)top_p * all;          // near enough to name the bin
    if (tid == 0) {
      sm.pick = 0;
      sm.digit = 0;
    }
    __syncthreads();
    int last = 0;                     // the last bin with tokens that starts below the goal
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (sm.bin.count[tid * kPer + j] && c < goal) last = tid * kPer + j;
      c += mass[j];
    }
    last = __reduce_max_sync(kFull, last);
    if (lane == 0) atomicMax(&sm.pick, last);
    // the border is in that bin, or next to its ends: from the bin with tokens before it to the
    // one after it
    int b0, b1;
    filled_around<kThreads>(sm, b0, b1);
    int n_range = sm.bin.count[sm.pick];
    n_range += b0 < sm.pick ? sm.bin.count[b0] : 0;
    n_range += b1 > sm.pick ? sm.bin.count[b1] : 0;
    bool found = false;
    if (sm.pick < kBins - 2 && n_range <= kList) {
      double above = 0.0, below = 0.0;
      for (int vi = s0 + lane; vi < s1; vi += 32) {
        float v[N];
        row.load(vi, v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float z;
          const int b = bin_of(v[j], z);
          const double w = weight(v[j]);
          if (b < b0) {
            above += w;
            if (w >= (double)min_p) kept_here += w;
          } else if (b > b1) {
            below += w;
          } else {
            sm.list[atomicAdd(&sm.n, 1)] = entry_of(key_of(v[j]), row.index(vi, j));
          }
        }
      }
      above = block_sum<kThreads>(above, sm.part);
      below = block_sum<kThreads>(below, sm.part);
      listed = border_in_list<kThreads>(weight, sm, sm.n, above, below, (double)top_p);
      found = listed > 0;
    } else if (sm.pick < kBins - 2) {
      // count the range by parts of its keys; `grain` low bits tell no two of the row's logits
      // apart, and a part is 2^shift of what is left of a key
      bits = __reduce_or_sync(kFull, bits);
      if (lane == 0) atomicOr(&sm.digit, bits);
      __syncthreads();
      const int grain = min(20, __ffs(sm.digit | 1u << 20) - 1);
      const uint32_t hi = (b0 ? key_of(__double2float_ru((double)top - (b0 - 0.05) / (double)scale)) : max_key) >> grain;
      const uint32_t lo = key_of(__double2float_rd((double)top - (b1 + 1.05) / (double)scale)) >> grain;
      int shift = 0;
      while ((hi - lo) >> shift >= kBins) ++shift;
      const auto part_of = [&](uint32_t key) { return (int)min((hi - (key >> grain)) >> shift, (uint32_t)kBins - 1); };
      for (int i = tid; i < kBins; i += kThreads) sm.bin.count[i] = 0;
      __syncthreads();
      double above = 0.0, below = 0.0;
      for (int vi = s0 + lane; vi < s1; vi += 32) {
        float v[N];
        row.load(vi, v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float z;
          const int b = bin_of(v[j], z);
          if (b >= b0 && b <= b1) {
            atomicAdd(&sm.bin.count[part_of(key_of(v[j]))], 1u);
            continue;
          }
          const double w = weight(v[j]);
          if (b < b0) {
            above += w;
            if (w >= (double)min_p) kept_here += w;
          } else {
            below += w;
          }
        }
      }
      above = block_sum<kThreads>(above, sm.part);
      below = block_sum<kThreads>(below, sm.part);
      // the key in the middle of a part (its only one where shift is 0)
      const auto key_in = [&](int p) {
        const uint32_t k = (hi - ((uint32_t)p << shift) - ((1u << shift) >> 1)) << grain;
        return k & 0x80000000u ? k : k | ((1u << grain) - 1);
      };
      mine = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int p = tid * kPer + j, count = sm.bin.count[p];
        mass[j] = count ? count * weight(value_of(key_in(p))) : 0.0;
        mine += mass[j];
      }
      block_scan<kThreads>(mine, 0, sm, c, unused, all, unused_all);
      c += above;
      all += above;                             // what lies before and in the range
      goal = (double)top_p * (all + below);
      if (tid == 0) sm.pick = -1;
      __syncthreads();
      last = -1;
      double start = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (sm.bin.count[tid * kPer + j] && c < goal) {
          last = tid * kPer + j;
          start = c;
        }
        c += mass[j];
      }
      const int warp_last = __reduce_max_sync(kFull, last);
      if (lane == 0) atomicMax(&sm.pick, warp_last);
      __syncthreads();
      const int part = sm.pick;
      int p0 = part, p1 = part;
      if (part >= 0) filled_around<kThreads>(sm, p0, p1);
      if (part >= 0 && all >= goal && shift == 0) {
        // equals at the border: kept while the mass before them is below the goal
        if (part == last) {
          const int count = sm.bin.count[part];
          const double d = (goal - start) / weight(value_of(key_in(part)));
          sm.ties_left = d >= (double)count ? count : max(1, (int)ceil(d));
        }
        __syncthreads();
        edge = key_in(part);
        n_edge = sm.ties_left;
        found = true;
        for (int vi = s0 + lane; vi < s1; vi += 32) {
          float v[N];
          row.load(vi, v);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint32_t key = key_of(v[j]);
            ties += key == edge;
            float z;
            if (key > edge && bin_of(v[j], z) >= b0) {
              const double w = weight(v[j]);
              if (w >= (double)min_p) kept_here += w;
            }
          }
        }
      } else if (part >= 0 && all >= goal) {
        double between = 0.0, after = 0.0;
        for (int vi = s0 + lane; vi < s1; vi += 32) {
          float v[N];
          row.load(vi, v);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            float z;
            const int b = bin_of(v[j], z);
            if (b < b0 || b > b1) continue;
            const uint32_t key = key_of(v[j]);
            const int p = part_of(key);
            if (p < p0) {
              const double w = weight(v[j]);
              between += w;
              if (w >= (double)min_p) kept_here += w;
            } else if (p > p1) {
              after += weight(v[j]);
            } else {
              const int at = atomicAdd(&sm.n, 1);
              if (at < kList) sm.list[at] = entry_of(key, row.index(vi, j));
            }
          }
        }
        between = block_sum<kThreads>(between, sm.part);
        after = block_sum<kThreads>(after, sm.part);
        if (sm.n <= kList)
          listed = border_in_list<kThreads>(weight, sm, sm.n, above + between, after + below, (double)top_p);
        found = listed > 0;
      }
    }
    have_sums = found;
    if (listed > 0) {
      // the border, its kept equals, and the segment's share of the list
      edge = entry_key(sm.sorted[listed - 1]);
      const int n = sm.n;
      int equal = 0;
      for (int i = lane; i < n; i += 32) {
        const int vi = (entry_index(sm.sorted[i]) + row.off) / N;
        const uint32_t key = entry_key(sm.sorted[i]);
        const bool here = vi >= s0 && vi < s1;
        equal += key == edge && i < listed;
        ties += key == edge && here;
        if (here && key > edge && sm.list_w.w[i] >= (double)min_p) kept_here += sm.list_w.w[i];
      }
      n_edge = __reduce_add_sync(kFull, equal);
    }
    if (!found) {
      __syncthreads();
      descend<kThreads>(row, weight, sm, true, top_k, top_p, edge, n_edge);
    }
  } else if (top_p < 1.f && !kByValues) {
    descend<kThreads>(row, weight, sm, true, top_k, top_p, edge, n_edge);
  }

  // ---- kept weight above the border, and equals of it, by segments of the vocabulary --------
  const double w_raw = edge ? weight(value_of(edge)) : 0.0;
  const double w_edge = w_raw >= (double)min_p ? w_raw : 0.0;
  // a logit below this is out by min_p without its weight (the bound's own rounding aside)
  float low_x = -CUDART_INF_F;
  if (min_p > 0.f && top < CUDART_INF_F) {
    const float low = (float)((double)top + (double)t * (log((double)min_p) - 1e-3));
    low_x = low - fabsf(low) * 1e-6f;
  }
  if (!have_sums) {
    kept_here = 0.0;
    ties = 0;
    for (int vi = s0 + lane; vi < s1; vi += 32) {
      float v[N];
      row.load(vi, v);
      if (!edge && min_p == 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) kept_here += weight(v[j]);
        continue;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t key = key_of(v[j]);
        if (key > edge) {
          if (v[j] >= low_x) {
            const double w = weight(v[j]);
            if (w >= (double)min_p) kept_here += w;
          }
        } else if (key == edge) {
          ++ties;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) kept_here += __shfl_xor_sync(kFull, kept_here, o);
  ties = __reduce_add_sync(kFull, ties);
  __syncthreads();
  if (lane == 0) {
    sm.part[warp] = kept_here;
    sm.ipart[warp] = ties;
  }
  __syncthreads();
  // every warp by itself: lane w has segment w.  The first segment past the target, or the last with
  // weight
  const int equals = lane < kWarps ? sm.ipart[lane] : 0, equals_before = warp_scan(equals) - equals;
  const double in_segment =
      lane < kWarps ? sm.part[lane] + min(max(n_edge - equals_before, 0), equals) * w_edge : 0.0;
  const double end = warp_scan(in_segment), total = __shfl_sync(kFull, end, 31), target = (double)u * total;
  const unsigned weighs = __ballot_sync(kFull, in_segment > 0.0);
  const unsigned beyond = __ballot_sync(kFull, in_segment > 0.0 && end > target);
  const int pick = beyond ? __ffs(beyond) - 1 : weighs ? 31 - __clz(weighs) : 0;
  const double start = __shfl_sync(kFull, end, max(pick - 1, 0));
  double base = pick ? start : 0.0;
  int left = max(n_edge - __shfl_sync(kFull, equals_before, pick), 0);

  // ---- the token: the whole block over its segment --------------------------------------------
  const int e0 = min(row.vectors, pick * seg), e1 = min(row.vectors, e0 + seg);
  for (int v0 = e0; v0 < e1; v0 += kThreads) {
    const int vi = v0 + tid;
    float v[N];
    double above = 0.0;
    int eq = 0;
    if (vi < e1) {
      row.load(vi, v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t key = key_of(v[j]);
        if (key > edge) {
          if (v[j] >= low_x) {
            const double w = weight(v[j]);
            if (w >= (double)min_p) above += w;
          }
        } else if (key == edge) {
          ++eq;
        }
      }
    }
    double a_before, a_all;
    int c_before, c_all;
    block_scan<kThreads>(above, eq, sm, a_before, c_before, a_all, c_all);
    const int mine = min(max(left - c_before, 0), eq);
    const double before = base + a_before + min(c_before, left) * w_edge;
    const double own_w = above + mine * w_edge;
    const unsigned live = __ballot_sync(kFull, own_w > 0.0);
    const unsigned hit = __ballot_sync(kFull, own_w > 0.0 && before + own_w > target);
    // first thread past the target; without one, the last that holds kept weight
    if (tid == 0) {
      sm.n = kThreads;
      sm.digit = 0;
    }
    __syncthreads();
    if (lane == 0 && hit) atomicMin(&sm.n, warp * 32 + __ffs(hit) - 1);
    if (lane == 0 && live) atomicMax(&sm.digit, (unsigned)(warp * 32 + 32 - __clz(live)));
    __syncthreads();
    const bool past = sm.n < kThreads;
    const int src = past ? sm.n : (int)sm.digit - 1;
    if (tid == src) {
      double c = before, w_at = 0.0;
      int at = -1, k = mine;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t key = key_of(v[j]);
        double w = 0.0;
        if (key > edge) {
          w = weight(v[j]);
          if (w < (double)min_p) w = 0.0;
        } else if (key == edge && k > 0) {
          --k;
          w = w_edge;
        }
        if (w > 0.0 && !(at >= 0 && c > target)) {
          at = row.index(vi, j);
          w_at = w;
          c += w;
        }
      }
      put_token(a, r, at, w_at / total);
    }
    if (past) return;
    base += a_all + min(c_all, left) * w_edge;
    left -= min(c_all, left);
    __syncthreads();
  }
}

// Rows that leave SMs free have 1024 threads each, two of 512 share an SM otherwise: 128 rows of 100003
// logits in fp32 with mixed filters took 112 us with 1024 threads and 140 us with 512; 1024 rows of 50000
// 214 and 193 us.
template <typename T, int kThreads> cudaError_t launch_rows(const SampleArgs &a, cudaStream_t st) {
  constexpr int kBytes = sizeof(T) == 2 ? (int)sizeof(ValueSmem) : 0;
  auto kernel = sample_kernel<T, kThreads>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<a.R, kThreads, kBytes, st>>>(a);
  return cudaGetLastError();
}

template <typename T> cudaError_t launch_type(const SampleArgs &a, cudaStream_t st) {
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return e;
  return a.R <= sms ? launch_rows<T, 1024>(a, st) : launch_rows<T, 512>(a, st);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int in_dtype, cudaStream_t st) {
  return in_dtype == TV_F32 ? launch_type<float>(a, st) : launch_type<__nv_bfloat16>(a, st);
}

}  // namespace tv
