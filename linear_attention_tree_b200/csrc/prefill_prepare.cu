// Prefill on tensor cores, first half: what a chunk's tokens are to one another, every chunk and head
// at once.  With cl the sum of log_a inside the chunk (64 tokens),
//     P[n][i] = exp(cl_n - cl_i) q_n.k_i  (i <= n),
//     L[n][i] = b_n exp(cl_n - cl_i) k_n.k_i  (i < n),   T = (I + L)^-1 diag(b)   (gated delta rule),
// into the workspace, for prefill_tc.cu, which carries the states from chunk to chunk.
//
// Persistent CTAs, three per SM, go through (chunk, head) items: warp 8 finds an item's sequence, brings
// its q and k by TMA and makes its gates, an item ahead; warps 0-7 compute.  (Without that an item's
// loads in a row are 8 us: 8 x 1000 tokens of scalar decay took 98 us in all with a CTA per item, 90 us
// so.)  [Q;K] K^T is one tcgen05 product (128 x 64) into tensor memory; a lane there is a row of P or
// of L.  T comes by the 16 x 16 diagonal blocks, by substitution in fp32, one warp each, then the
// blocks below them by products of 16 x 16 blocks: too small for tcgen05 (128 rows) and, as
// multiply-adds, bound by the registers' fill from shared memory (128 bytes a cycle), so they are
// warp-level tf32 products of high and low halves, which halved all shared-memory reads of the kernel.
// The kernel runs apart from the chain over chunks, whose SMs it kept busy when both were one: 1 x 8192
// tokens of 32 heads took 963 us then, 671 us as two kernels.
// 2560 items (5120 tokens of 32 heads) take 51 us, 4096 (those 8192 tokens) 75 us: 187 MB at 2.5 TB/s, the
// shared-memory pipe 70% busy, which bounds it, issue slots 46%.
//
// Every wait is bounded: one that runs out records TV_ERR_TIMEOUT and ends the CTA.
#include <algorithm>
#include <climits>

#include "prefill_tc.cuh"

namespace tv {
namespace {

using namespace prefill;

constexpr int kWarps = 8;                    // computing warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kPerSm = 3;
constexpr int kLd = 68;                      // row of the fp32 work matrices
constexpr uint32_t kSpinLimit = 1u << 22;

// The work matrices of an item, over its [Q ; K] once their product is there.
struct Matrices {
  float L[kC][kLd];      // strictly lower; T's diagonal blocks over its own; products of blocks in the
                         // blocks above the diagonal
  float Tt[kC][kLd];     // P, then T transposed
};
static_assert(sizeof(Matrices) >= 2 * kHalf && sizeof(Matrices) % 1024 == 0, "the matrices cover the tiles");
struct Item {
  int slot, h, rows;                         // slot -1: no more
  __align__(16) float clh[kC];               // cl in powers of two, as a pair
  float cll[kC];
  float end[kC];                             // exp(cl at the end of the block of 16 - cl)
  float b[kC];
};
struct Work {
  Item item[2];
  unsigned long long full[2], empty[2], done;
  uint32_t tmem;
  int no_tile, no_product;                   // a wait for one has run out
};
constexpr int kOffWork = 2 * (int)sizeof(Matrices);
constexpr int kSmemBytes = kOffWork + (int)sizeof(Work) + 1024;

// D += A B for 16 x 8 tf32 tiles of one warp (lane: g = lane / 4, t = lane % 4): a = A[g][t], A[g+8][t],
// A[g][t+4], A[g+8][t+4]; b = B[t][g], B[t+4][g]; d = D[g][2t], D[g][2t+1], D[g+8][2t], D[g+8][2t+1].
__device__ __forceinline__ void mma_16x8x8(float (&d)[4], const float (&a)[4], float b0, float b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// acc += a 16 x 16 block (rows of kLd at A) times eight columns (each along b, `ld` apart), as pairs
// of tf32: high by high, high by low and low by high.  High parts are rounded (11 bits), low ones
// take what the product keeps of them (10 bits at least): 2^-21.  A lane's four values of k are
// neighbours, which renames the k of the tiles alike on both sides.
__device__ __forceinline__ void block_product(float (&acc)[4], const float *A, const float *b, int ld, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float4 p = *reinterpret_cast<const float4 *>(A + g * kLd + 4 * t);
  const float4 q = *reinterpret_cast<const float4 *>(A + (g + 8) * kLd + 4 * t);
  const float4 y = *reinterpret_cast<const float4 *>(b + g * ld + 4 * t);
  const float a[2][4] = {{p.x, q.x, p.y, q.y}, {p.z, q.z, p.w, q.w}}, v[2][2] = {{y.x, y.y}, {y.z, y.w}};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float hi[4], low[4], vh[2], vl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = tf32_round(a[s][i]);
      low[i] = a[s][i] - hi[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      vh[i] = tf32_round(v[s][i]);
      vl[i] = v[s][i] - vh[i];
    }
    mma_16x8x8(acc, low, vh[0], vh[1]);
    mma_16x8x8(acc, hi, vl[0], vl[1]);
    mma_16x8x8(acc, hi, vh[0], vh[1]);
  }
}

// Eight columns of a block, transposed to rows of `ld` at `to`.
__device__ __forceinline__ void store_columns(float *to, int ld, const float (&acc)[4], float sign, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int e = 0; e < 4; ++e) to[(2 * t + (e & 1)) * ld + g + 8 * (e >> 1)] = sign * acc[e];
}

// Column c of product i, in a block of L above the diagonal.
__device__ __forceinline__ float *y_at(Matrices &m, int i, int c) {
  return i < 3 ? &m.L[c][16 * (i + 1)] : &m.L[16 + c][32];
}

// m.Tt = the transpose of (I + L)^-1 for the unit lower triangular system in m.L: the four diagonal
// blocks of 16 by substitution; blocks (1, 0) and (3, 2), T_iJ = -T_ii (L_iJ T_JJ), which complete the
// diagonal blocks of 32; then the block of 32 below them, -T' (L' T'') with all eight warps.
__device__ __forceinline__ void invert(Matrices &m, int w, int lane) {
  if (w < 4) {
    const int col = lane & 15, half = lane >> 4;
    float x[16];
    float *D = &m.L[16 * w][16 * w];
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      float s[4] = {n == col ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < n; i += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(D + n * kLd + i);
        s[0] = fmaf(-l.x, x[i], s[0]);
        if (i + 1 < n) s[1] = fmaf(-l.y, x[i + 1], s[1]);
        if (i + 2 < n) s[2] = fmaf(-l.z, x[i + 2], s[2]);
        if (i + 3 < n) s[3] = fmaf(-l.w, x[i + 3], s[3]);
      }
      x[n] = (s[0] + s[1]) + (s[2] + s[3]);
    }
    __syncwarp();
    // both halves hold the column: each writes eight rows
    const int row = 8 * half;
    float y[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      y[n] = half ? x[n + 8] : x[n];
      D[(row + n) * kLd + col] = y[n];
    }
    float4 *tt = reinterpret_cast<float4 *>(&m.Tt[16 * w + col][16 * w + row]);
    tt[0] = make_float4(y[0], y[1], y[2], y[3]);
    tt[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
  group_sync(1, kWarps * 32);
  const int c0 = 8 * (w & 1);                     // eight columns of a block to a warp
  float pair[4] = {};                             // T_10 or T_32
  if (w < 4) {
    const int b = w >> 1, J = 2 * b, i = J + 1;
    float acc[4] = {};
    block_product(acc, &m.L[16 * i][16 * J], &m.Tt[16 * J + c0][16 * J], kLd, lane);
    store_columns(y_at(m, b, c0), kLd, acc, 1.f, lane);
    __syncwarp();
    block_product(pair, &m.L[16 * i][16 * i], y_at(m, b, c0), kLd, lane);
    store_columns(&m.Tt[16 * J + c0][16 * i], kLd, pair, -1.f, lane);
  }
  group_sync(1, kWarps * 32);
  if (w == 2 || w == 3) {
    // T_32 by rows too, over L_32, which both of these warps read whole before the barrier; it is read
    // in the last step
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; ++e) m.L[48 + g + 8 * (e >> 1)][32 + c0 + 2 * t + (e & 1)] = -pair[e];
  }
  const int I = 2 + (w >> 2), J = w >> 1 & 1;
  {
    float acc[4] = {};
    for (int k = J; k < 2; ++k)
      block_product(acc, &m.L[16 * I][16 * k], &m.Tt[16 * J + c0][16 * k], kLd, lane);
    store_columns(y_at(m, w >> 1, c0), kLd, acc, 1.f, lane);
  }
  group_sync(1, kWarps * 32);
  {
    float out[4] = {};
    for (int k = 2; k <= I; ++k)
      block_product(out, &m.L[16 * I][16 * k], y_at(m, 2 * (k - 2) + J, c0), kLd, lane);
    store_columns(&m.Tt[16 * J + c0][16 * I], kLd, out, -1.f, lane);
  }
}

// The blocks of a work matrix to the workspace: block (i, j) from rows 16 i, columns 16 j of m, or
// (transposed) from rows 16 j, columns 16 i, with every row scaled.
template <bool kTransposed>
__device__ __forceinline__ void write_blocks(float *to, const float (*m)[kLd], const float *scale) {
  for (int e = threadIdx.x; e < kPart / 4; e += kWarps * 32) {
    const int b = e >> 6, I = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3, J = b - I * (I + 1) / 2;
    const int row = 16 * (kTransposed ? J : I) + (e >> 2 & 15), col = 16 * (kTransposed ? I : J) + 4 * (e & 3);
    float4 x = *reinterpret_cast<const float4 *>(&m[row][col]);
    if (kTransposed) {
      const float f = scale[row];
      x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
    }
    reinterpret_cast<float4 *>(to)[e] = x;
  }
}

template <bool kGdn>
__global__ void __launch_bounds__(kThreads, kPerSm)
    prepare_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   SequenceArgs a, int items) {
  extern __shared__ unsigned char smem_dyn[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Work &wk = *reinterpret_cast<Work *>(sm + kOffWork);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, H = a.H;
  const uint32_t sbase = ptx::smem_addr(sm), done = ptx::smem_addr(&wk.done);
  const uint32_t full = ptx::smem_addr(&wk.full[0]), empty = ptx::smem_addr(&wk.empty[0]);
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(full + 8 * b, 1);
      ptx::mbar_init(empty + 8 * b, kWarps);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_mbar_init();
    wk.no_tile = wk.no_product = 0;
  }
  if (w == 0) {
    ptx::tmem_alloc(ptx::smem_addr(&wk.tmem), kC);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = wk.tmem;

  bool late = false;
  if (w == kWarps) {
    // ==== items, their tiles and gates ===========================================================
    const bool one = elect_one();
    int it = 0;
    for (int i = blockIdx.x; i < items && !late; i += gridDim.x) {
      const int slot = i / H, h = i % H, kh = qk_head(h, H, a.Hk);
      // the sequence that the slot belongs to, if one does: of several (offsets that do not rise)
      // only the first can be a good one
      int s = INT_MAX;
      for (int x = lane; x < a.B; x += 32) {
        int lo, n;
        const bool in = sequence_range(a.offsets, x, a.T, a.max_len, lo, n);
        const int c = slot - (lo / kC + x);
        if (in && c >= 0 && c * kC < n) s = min(s, x);
      }
      s = __reduce_min_sync(0xffffffffu, s);
      if (s == INT_MAX) continue;
      const int lo = a.offsets[s], n = a.offsets[s + 1] - lo, c = slot - (lo / kC + s);
      if (!__all_sync(0xffffffffu, sequence_rises(a.offsets, s, lo, lane, 32))) continue;
      const int first = lo + c * kC, rows = min(kC, n - c * kC), buf = it & 1;
      double x[2];
      float b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        const size_t at = (size_t)(first + t) * H + h;
        x[e] = t < rows ? log2_decay(a.log_a[at]) : 0.0;
        b[e] = kGdn && t < rows ? a.b[at] : 0.f;
      }
      if (it >= 2 && !ptx::mbar_wait_bounded(empty + 8 * buf, (it >> 1) - 1 & 1, kSpinLimit)) {
        late = true;
        break;
      }
      if (one) {
        ptx::fence_proxy_async_smem();           // the matrices there have been read
        const uint32_t to = sbase + buf * (int)sizeof(Matrices);
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(full + 8 * buf),
                     "r"(2 * kHalf)
                     : "memory");
        for (int half = 0; half < 2; ++half) {
          ptx::tma_load_3d(to + half * kHalf + kKRow, &tm_k, full + 8 * buf, half * 64, kh, first);
          ptx::tma_load_3d(to + half * kHalf, &tm_q, full + 8 * buf, half * 64, kh, first);
        }
      }
      Item &m = wk.item[buf];
      const double sum = prefix(x), end = __shfl_sync(0xffffffffu, sum, lane | 7);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const double cl = e ? sum : sum - x[1];
        const int t = 2 * lane + e;
        const float hi = (float)cl;
        m.clh[t] = hi;
        m.cll[t] = (float)(cl - (double)hi);
        m.end[t] = fminf(exp2f((float)(end - cl)), 3e38f);
        m.b[t] = b[e];
      }
      if (one) {
        m.slot = slot;
        m.h = h;
        m.rows = rows;
      }
      __syncwarp();
      if (one) ptx::mbar_arrive(full + 8 * buf);
      ++it;
    }
    // the last tile that was asked for has come before the CTA ends; then the end of the items
    const int buf = it & 1;
    if (it > 0) ptx::mbar_wait_bounded(full + 8 * (buf ^ 1), (it - 1) >> 1 & 1, kSpinLimit);
    if (!late && it >= 2) late = !ptx::mbar_wait_bounded(empty + 8 * buf, (it >> 1) - 1 & 1, kSpinLimit);
    if (!late && one) {
      wk.item[buf].slot = -1;
      ptx::mbar_arrive(full + 8 * buf);
    }
    __syncwarp();
  } else {
    for (int it = 0;; ++it) {
      const int buf = it & 1;
      // one warp waits, the others at the barrier behind it
      if (w == 0 && !ptx::mbar_wait_bounded(full + 8 * buf, it >> 1 & 1, kSpinLimit)) wk.no_tile = 1;
      group_sync(1, kWarps * 32);
      const Item &t = wk.item[buf];
      if (wk.no_tile || t.slot < 0) break;
      unsigned char *tile = sm + buf * sizeof(Matrices);
      Matrices &m = *reinterpret_cast<Matrices *>(tile);
      const int rows = t.rows;
      if (rows < kC) {
        // rows past the sequence may hold anything: as keys they are zero (their own rows are not used)
        for (int e = tid; e < (kC - rows) * 16; e += kWarps * 32) {
          const int r = rows + (e >> 4), x = e & 15;
          *reinterpret_cast<uint4 *>(tile + (x >> 3) * kHalf + kKRow + r * 128 + (x & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        group_sync(1, kWarps * 32);
      }
      if (w == 0) {
        const bool one = elect_one();
        const uint64_t q = ptx::smem_desc_sw128(ptx::smem_addr(tile), 1024), k = q + (kKRow >> 4);
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t step = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          mma_f16(one, tmem, q + step, k + step, ptx::idesc_bf16_f32(128, kC), kk > 0);
        }
        mma_done(one, done);
        if (!ptx::mbar_wait_bounded(done, it & 1, kSpinLimit)) wk.no_product = 1;
      }
      group_sync(1, kWarps * 32);
      if (wk.no_product) break;
      ptx::tc_fence_after();
      float x[32];
      const int hf = w >> 2;                          // columns 32 hf
      tmem_load(tmem + ((uint32_t)(32 * (w & 3)) << 16) + 32 * hf, x);
      // Decay ratios: inside a diagonal block of 16 one by one; before it as the product of exp(cl_row
      // - cl at the end of the column's block) and `end` of the column (both at most 1 for decays).
      // Blocks behind the diagonal are not used.
      const int row = (32 * w + lane) & 63;           // warps 0, 1 and 4, 5: q rows; others: k rows
      const bool is_k = w & 2;
      const float clh = t.clh[row], cll = t.cll[row], scale = is_k ? t.b[row] : 1.f;
      const int last = is_k ? row - 1 : row;
      const bool diagonal = hf == (w & 1);            // of some of the warp's rows
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        const int J = 2 * hf + jb;
        const float before =
            J < row >> 4 ? scale * pow2((clh - t.clh[16 * J + 15]) + (cll - t.cll[16 * J + 15])) : 0.f;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int i = 16 * J + j, at = 16 * jb + j;
          const float4 end = *reinterpret_cast<const float4 *>(&t.end[i]);
          const float f[4] = {before * end.x, before * end.y, before * end.z, before * end.w};
          if (diagonal) {
            const float4 ch = *reinterpret_cast<const float4 *>(&t.clh[i]);
            const float4 cl = *reinterpret_cast<const float4 *>(&t.cll[i]);
            const float d[4] = {(clh - ch.x) + (cll - cl.x), (clh - ch.y) + (cll - cl.y),
                                (clh - ch.z) + (cll - cl.z), (clh - ch.w) + (cll - cl.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float own = i + e <= last ? scale * pow2(d[e]) * x[at + e] : 0.f;
              x[at + e] = J == row >> 4 ? own : f[e] * x[at + e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[at + e] *= f[e];
          }
        }
      }
      // rows of P and L into shared memory (the tiles there are done with), P to the workspace
      float(*to)[kLd] = is_k ? m.L : m.Tt;
      if (kGdn || !is_k) {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4 *>(&to[row][32 * hf + i]) =
              make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
      ptx::tc_fence_before();
      group_sync(1, kWarps * 32);
      float *out = slot_at(a, kGdn, t.slot, t.h);
      write_blocks<false>(out, m.Tt, nullptr);
      if (kGdn) {
        group_sync(1, kWarps * 32);
        invert(m, w, lane);
        group_sync(1, kWarps * 32);
        write_blocks<true>(out + kPart, m.Tt, t.b);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * buf);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  if (__syncthreads_or(late || wk.no_tile || wk.no_product) && tid == 0) set_status(a.ws, TV_ERR_TIMEOUT, 0);
  if (w == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kC);
  }
}

template <bool kGdn> cudaError_t launch(const SequenceArgs &a, cudaStream_t st) {
  CUtensorMap tq, tk;
  if (!make_node_map(&tq, a.q, a.Hk, a.T, kC) || !make_node_map(&tk, a.k, a.Hk, a.T, kC))
    return cudaErrorInvalidValue;
  auto kernel = prepare_kernel<kGdn>;
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int items = (int)(slots(a.T, a.B) * a.H);
  kernel<<<std::min(items, sms * kPerSm), kThreads, kSmemBytes, st>>>(tq, tk, a, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_prepare(const SequenceArgs &a, int mode, cudaStream_t st) {
  return mode == TV_MODE_GDN ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace tv
