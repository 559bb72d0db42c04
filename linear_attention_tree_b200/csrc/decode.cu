// One token of every sequence through the recurrence, the state updated in one pass:
//     p = S k,  u = b (v - a p)  (scalar decay: u = v),  S' = a S + u k^T,  o = S' q .
//
// The rows of S are independent given k and q, and the state is read and written once:
// 2 * dv * dk * 4 bytes per (sequence, head), which bounds large batches.  Eight lanes hold a
// row (NK float4 each, so a warp's load covers four rows in whole 128-byte segments), and
// each dot product costs three shuffles.  A CTA takes kRows rows of one state, all of its
// loads in flight before the first product.
// 128 sequences of 32 heads, dk = dv = 128: 82 us for 544 MB (6.6 TB/s, all of the measured copy
// bandwidth).  32 sequences: 27 us for 136 MB (5.0 TB/s; a plain copy of the states takes 28.7 us): four
// waves of CTAs, of which the first waits for its loads and the last for its stores, with DRAM at 30% and
// issue slots at 28% in between since most of the writes stay in L2.
#include "serving.cuh"

namespace tv {
namespace {

constexpr int kThreads = 128;
constexpr int kRowsPerThread = 2;
constexpr int kRows = kThreads / 8 * kRowsPerThread;   // state rows per CTA

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
// Sum over the eight lanes of a row.
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

template <typename Tin, typename Tout, bool kGdn, int NK>
__global__ void __launch_bounds__(kThreads) decode_kernel(SequenceArgs a) {
  const int H = a.H, dk = a.dk, dv = a.dv;
  const int slices = (dv + kRows - 1) / kRows;
  const int item = blockIdx.x / slices, r0 = (blockIdx.x % slices) * kRows;
  const int s = item / H, h = item % H, kh = qk_head(h, H, a.Hk);
  const int lane8 = threadIdx.x & 7, group = threadIdx.x >> 3;
  const size_t state = (size_t)item * dv * dk;

  float4 S[kRowsPerThread][NK];
#pragma unroll
  for (int r = 0; r < kRowsPerThread; ++r) {
    const int row = r0 + group + r * (kThreads / 8);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int col = 4 * (lane8 + 8 * i);
      S[r][i] = row < dv && col < dk
                    ? __ldcs(reinterpret_cast<const float4 *>(a.S_in + state + (size_t)row * dk + col))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  const Tin *kg = static_cast<const Tin *>(a.k) + ((size_t)s * a.Hk + kh) * dk;
  const Tin *qg = static_cast<const Tin *>(a.q) + ((size_t)s * a.Hk + kh) * dk;
  float4 k[NK], q[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int col = 4 * (lane8 + 8 * i);
    k[i] = q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < dk) {
      k[i] = load4(kg + col);
      q[i] = load4(qg + col);
    }
  }
  const float decay = expf(a.log_a[item]), b = kGdn ? a.b[item] : 0.f;
  if (decay == 0.f) {                  // starts afresh, also from NaN and infinity
#pragma unroll
    for (int r = 0; r < kRowsPerThread; ++r)
#pragma unroll
      for (int i = 0; i < NK; ++i) S[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

#pragma unroll
  for (int r = 0; r < kRowsPerThread; ++r) {
    const int row = r0 + group + r * (kThreads / 8);
    const size_t at = (size_t)item * dv + row;
    float u = row < dv ? to_f32(static_cast<const Tin *>(a.v)[at]) : 0.f;
    if (kGdn) {
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < NK; ++i) p = dot4(S[r][i], k[i], p);
      u = b * (u - decay * sum8(p));
    }
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      S[r][i].x = fmaf(u, k[i].x, decay * S[r][i].x);
      S[r][i].y = fmaf(u, k[i].y, decay * S[r][i].y);
      S[r][i].z = fmaf(u, k[i].z, decay * S[r][i].z);
      S[r][i].w = fmaf(u, k[i].w, decay * S[r][i].w);
      o = dot4(S[r][i], q[i], o);
    }
    o = sum8(o);
    if (row < dv) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int col = 4 * (lane8 + 8 * i);
        if (col < dk)
          __stcs(reinterpret_cast<float4 *>(a.S_out + state + (size_t)row * dk + col), S[r][i]);
      }
      if (lane8 == 0) static_cast<Tout *>(a.out)[at] = from_f32<Tout>(o);
    }
  }
}

template <typename Tin, typename Tout, bool kGdn>
cudaError_t launch(const SequenceArgs &a, cudaStream_t st) {
  const int slices = (a.dv + kRows - 1) / kRows;
  const unsigned grid = (unsigned)a.B * a.H * slices;
  switch ((a.dk + 31) / 32) {
    case 1: decode_kernel<Tin, Tout, kGdn, 1><<<grid, kThreads, 0, st>>>(a); break;
    case 2: decode_kernel<Tin, Tout, kGdn, 2><<<grid, kThreads, 0, st>>>(a); break;
    case 3: decode_kernel<Tin, Tout, kGdn, 3><<<grid, kThreads, 0, st>>>(a); break;
    default: decode_kernel<Tin, Tout, kGdn, 4><<<grid, kThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t launch_mode(const SequenceArgs &a, int mode, cudaStream_t st) {
  return mode == TV_MODE_GDN ? launch<Tin, Tout, true>(a, st) : launch<Tin, Tout, false>(a, st);
}

}  // namespace

cudaError_t launch_decode_step(const SequenceArgs &a, int mode, int in_dtype, int out_dtype,
                               cudaStream_t st) {
  if (in_dtype == TV_F32) return launch_mode<float, float>(a, mode, st);
  if (out_dtype == TV_F32) return launch_mode<__nv_bfloat16, float>(a, mode, st);
  return launch_mode<__nv_bfloat16, __nv_bfloat16>(a, mode, st);
}

}  // namespace tv
