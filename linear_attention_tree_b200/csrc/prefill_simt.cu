// Whole prompts through the recurrence, token by token on CUDA cores, every shape and type:
//     S_t = a_t S_{t-1}(I - b_t k_t k_t^T) + b_t v_t k_t^T  (scalar: S_t = a_t S_{t-1} + v_t k_t^T),
//     o_t = S_t q_t .
//
// The rows of S are independent given k and q: eight lanes hold a row in registers for the
// whole prompt (NK float4 each), and a CTA of 128 threads holds 16 rows of one (sequence,
// head).  A token costs the chain u -> S' -> S' k (the next token's dot product, in four running
// sums, and three shuffles); o = S' q is formed beside it.  Tokens arrive in double-buffered
// tiles of kTile by cp.async in their own type and are widened as they are read.  fp32 throughout.
// Bound by that chain where CTAs are few, 0.2 us a token (16 heads, 256 tokens: 62 us, 2048: 445 us; as
// one running sum before the update the dot product made it nearly twice that), by instructions where they
// are many (32 x 64 tokens, 32 heads: 450 us).
#include "serving.cuh"
#include "tc_ptx.cuh"

namespace tv {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = kThreads / 8;     // state rows per CTA
constexpr int kTile = 16;               // tokens per shared-memory tile

template <typename Tin> struct __align__(16) Tile {
  Tin k[kTile][128];
  Tin q[kTile][128];
  Tin v[kTile][kRows];
  float la[kTile];
  float b[kTile];
};

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
// Four running sums (a single one would make a chain of the whole row).
__device__ __forceinline__ void dot4(float4 a, float4 b, float4 &s) {
  s.x = fmaf(a.x, b.x, s.x);
  s.y = fmaf(a.y, b.y, s.y);
  s.z = fmaf(a.z, b.z, s.z);
  s.w = fmaf(a.w, b.w, s.w);
}
__device__ __forceinline__ float sum4(float4 s) { return (s.x + s.y) + (s.z + s.w); }
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_addr(dst)), "l"(src)
               : "memory");
}

template <typename Tin, bool kGdn>
__device__ __forceinline__ void fetch(const SequenceArgs &a, Tile<Tin> &t, size_t first, int n, int h,
                                      int kh, int r0) {
  constexpr int kVec = 16 / sizeof(Tin);            // elements per 16-byte copy
  const int dk = a.dk, per_row = dk / kVec;
  const Tin *q = static_cast<const Tin *>(a.q), *k = static_cast<const Tin *>(a.k);
  for (int e = threadIdx.x; e < n * per_row; e += kThreads) {
    const int i = e / per_row, c = (e % per_row) * kVec;
    const size_t row = ((first + i) * a.Hk + kh) * dk + c;
    copy16(&t.k[i][c], k + row);
    copy16(&t.q[i][c], q + row);
  }
  constexpr int kVr = kRows / kVec;
  const Tin *v = static_cast<const Tin *>(a.v);
  for (int e = threadIdx.x; e < n * kVr; e += kThreads) {
    const int i = e / kVr, c = (e % kVr) * kVec;
    copy16(&t.v[i][c], v + ((first + i) * a.H + h) * a.dv + r0 + c);
  }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    copy4(&t.la[i], a.log_a + (first + i) * a.H + h);
    if (kGdn) copy4(&t.b[i], a.b + (first + i) * a.H + h);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename Tin, typename Tout, bool kGdn, int NK>
__global__ void __launch_bounds__(kThreads) prefill_kernel(SequenceArgs a) {
  __shared__ Tile<Tin> tile[2];
  __shared__ float o_tile[2][kTile][kRows];
  const int H = a.H, dk = a.dk, dv = a.dv, slices = dv / kRows;
  const int item = blockIdx.x / slices, r0 = (blockIdx.x % slices) * kRows;
  const int s = item / H, h = item % H, kh = qk_head(h, H, a.Hk);
  const int lane8 = threadIdx.x & 7, group = threadIdx.x >> 3;
  int lo, n;
  const bool in = sequence_range(a.offsets, s, a.T, a.max_len, lo, n);
  if (!__syncthreads_and(in && sequence_rises(a.offsets, s, lo, threadIdx.x, kThreads))) {
    if (threadIdx.x == 0) set_status(a.ws, TV_ERR_BAD_TREE, s);
    return;
  }
  const float *S_in = a.S_in;
  if (n > 0) {
    // a first decay of zero starts afresh, also from NaN and infinity
    if (expf(a.log_a[(size_t)lo * H + h]) == 0.f) S_in = nullptr;
    fetch<Tin, kGdn>(a, tile[0], lo, min(kTile, n), h, kh, r0);
  }

  const size_t state = (size_t)item * dv * dk + (size_t)(r0 + group) * dk;
  float4 S[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int col = 4 * (lane8 + 8 * i);
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (S_in && col < dk) S[i] = *reinterpret_cast<const float4 *>(S_in + state + col);
  }

  Tout *out = static_cast<Tout *>(a.out);
  for (int t0 = 0, buf = 0; t0 < n; t0 += kTile, buf ^= 1) {
    const int m = min(kTile, n - t0);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                  // this tile is here; the other one has been read
    if (t0 + kTile < n)
      fetch<Tin, kGdn>(a, tile[buf ^ 1], (size_t)lo + t0 + kTile, min(kTile, n - t0 - kTile), h, kh, r0);
    const Tile<Tin> &tl = tile[buf];
    const auto load = [&](const Tin *row, float4 (&x)[NK]) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int col = 4 * (lane8 + 8 * i);
        x[i] = col < dk ? load4(row + col) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    float4 k[NK], sp = make_float4(0.f, 0.f, 0.f, 0.f);
    load(tl.k[0], k);
#pragma unroll
    for (int i = 0; i < NK; ++i) dot4(S[i], k[i], sp);
    float p = kGdn ? sum8(sum4(sp)) : 0.f, decay = expf(tl.la[0]);
#pragma unroll 2
    for (int t = 0; t < m; ++t) {
      const int next = min(t + 1, m - 1);
      float4 q[NK], kn[NK];
      load(tl.q[t], q);
      load(tl.k[next], kn);
      const float decay_next = expf(tl.la[next]);
      float u = to_f32(tl.v[t][group]);
      if (kGdn) u = tl.b[t] * (u - decay * p);
      float4 so = make_float4(0.f, 0.f, 0.f, 0.f);
      sp = so;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        S[i].x = fmaf(u, k[i].x, decay * S[i].x);
        S[i].y = fmaf(u, k[i].y, decay * S[i].y);
        S[i].z = fmaf(u, k[i].z, decay * S[i].z);
        S[i].w = fmaf(u, k[i].w, decay * S[i].w);
        if (kGdn) dot4(S[i], kn[i], sp);
        dot4(S[i], q[i], so);
        k[i] = kn[i];
      }
      const float o = sum8(sum4(so));
      if (kGdn) p = sum8(sum4(sp));
      decay = decay_next;
      if (lane8 == 0) o_tile[buf][t][group] = o;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < m * kRows; e += kThreads)
      out[((size_t)(lo + t0 + e / kRows) * H + h) * dv + r0 + e % kRows] =
          from_f32<Tout>(o_tile[buf][e / kRows][e % kRows]);
  }
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int col = 4 * (lane8 + 8 * i);
    if (col < dk) *reinterpret_cast<float4 *>(a.S_out + state + col) = S[i];
  }
}

template <typename Tin, typename Tout, bool kGdn>
cudaError_t launch(const SequenceArgs &a, cudaStream_t st) {
  const unsigned grid = (unsigned)a.B * a.H * (a.dv / kRows);
  switch ((a.dk + 31) / 32) {
    case 1: prefill_kernel<Tin, Tout, kGdn, 1><<<grid, kThreads, 0, st>>>(a); break;
    case 2: prefill_kernel<Tin, Tout, kGdn, 2><<<grid, kThreads, 0, st>>>(a); break;
    case 3: prefill_kernel<Tin, Tout, kGdn, 3><<<grid, kThreads, 0, st>>>(a); break;
    default: prefill_kernel<Tin, Tout, kGdn, 4><<<grid, kThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t launch_mode(const SequenceArgs &a, int mode, cudaStream_t st) {
  return mode == TV_MODE_GDN ? launch<Tin, Tout, true>(a, st) : launch<Tin, Tout, false>(a, st);
}

}  // namespace

cudaError_t launch_prefill_simt(const SequenceArgs &a, int mode, int in_dtype, int out_dtype,
                                cudaStream_t st) {
  if (in_dtype == TV_F32) return launch_mode<float, float>(a, mode, st);
  if (out_dtype == TV_F32) return launch_mode<__nv_bfloat16, float>(a, mode, st);
  return launch_mode<__nv_bfloat16, __nv_bfloat16>(a, mode, st);
}

}  // namespace tv
