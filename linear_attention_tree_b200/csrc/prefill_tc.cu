// Whole prompts through the recurrence on tensor cores: bf16 q / k / v, dk = dv = 128, gated
// delta rule or scalar decay, fp32 states.
//
// A sequence is taken in chunks of 64 tokens.  With cl the sum of log_a inside the chunk,
// gamma = exp(cl), S the state before it and g = gamma of its last token, the recurrence's
// closed form is
//     R_n = v_n - gamma_n S k_n,    U = T R,  T = (I + L)^-1 diag(b),
//     L[n][i] = b_n exp(cl_n - cl_i) k_n.k_i  (i < n),
//     o_n = gamma_n S q_n + sum_{i <= n} P[n][i] u_i,  P[n][i] = exp(cl_n - cl_i) q_n.k_i,
//     S' = g S + sum_i exp(cl_last - cl_i) u_i k_i^T          (scalar decay: U = V).
// Everything is kept transposed as in the verify kernels: tensor-memory lane = value row v.
//
// Precision.  States are fp32 and every product is as good: a bf16 operand (k, q) meets an fp32 one cut
// into three bf16 pieces of 8 bits (exact), T and R meet as pairs of tf32 (22 bits; the product of the
// two low parts, 2^-22 and less, is left out), U and P as three bf16 pieces each (products of 2^-24
// and less are left out).  out in bf16 is out in fp32 rounded once: with two pieces of S for S Q^T and one tf32
// product U P^T for it, 3% of its values were a step off and the three times below 5 to 6% shorter.
// Decay ratios are powers of two of a difference of sums kept as an fp32 pair.
//
// P and T of every chunk come from prefill_prepare.cu through the workspace; the states' chain runs
// here, one CTA of 22 warps per (sequence, head), one per SM.  The chain of a chunk is
//     S -> [S K^T] -> R -> [R T^T] -> U -> [U~ K] -> S'          ([..] tensor core),
// and everything else is done beside it:
//   warps 0-15  the chain: S in registers (lane v, 32 of 128 columns each), its pieces, R, U and
//               its pieces into tensor memory; the previous chunk's o = gamma S q + P U stored.
//   warps 16-19 T and P of the next chunk from the workspace's blocks into operand tiles.
//   warp 20     the gates, and the copies (TMA, two buffers of each kind), a chunk or two ahead.
//   warp 21     the MMAs: S K^T, R T^T, S Q^T, U~ K, U P^T.
// Tensor memory (512 columns): [0,192) the pieces of S, D = U~ K over [0,128); [192,256) S K^T,
// then U, then low pieces of U; [256,320) S Q^T; [320,448) R as two tf32 halves, then the pieces of
// U~ and the high piece of U; [448,512) U P^T.
// Rows of a last partial chunk past the sequence are zeroed in shared memory (k and v), so that
// they add nothing.
//
// What bounds it is the chain: 8,100 cycles a chunk (4.6 us), of which the three products on it are
// 2,650 back to back (24 + 24 MMAs of 37 cycles, 12 of 74); the rest is the chain warps' own work on
// 128 x 128 values of S and 128 x 64 of R and U at half of the issue slots, and the output's products.
// One prompt of 8192 tokens, 32 heads, has 32 chains of 128 chunks: 595 us here, 75 us in
// prefill_prepare.cu (floor of the bytes: 41 us).  16 ragged prompts of 16384 tokens in all: 505 us with it
// (floor 72 us), 8 x 1000 tokens of scalar decay, 16 heads: 95 us (floor 23 us).  Sixteen chain warps
// instead of eight (latency), U~ and S handed over piece by piece and o stored while R T^T is computed
// shortened a chunk by 1,700 cycles.  22 warps leave 80 registers a thread, of which the chain spills 20
// to 25.
//
// Every wait is bounded: one that runs out records TV_ERR_TIMEOUT on the status word and ends the
// CTA after its copies and MMAs (bounded again).
#include "prefill_tc.cuh"

namespace tv {
namespace {

using namespace prefill;

constexpr int kChain = 16;                   // chain warps
constexpr int kPrep = 4;                     // warps that place T and P
constexpr int kThreads = (kChain + kPrep + 2) * 32;
constexpr uint32_t kSpinLimit = 1u << 22;

// tensor memory columns
constexpr uint32_t kColS = 0, kColD = 0, kColSK = 192, kColSQ = 256, kColR = 320, kColUP = 448;
constexpr uint32_t kColUt = 320, kColU = 416;

// dynamic shared memory, from a 1024-byte aligned base
constexpr int kTileBytes = 2 * kHalf + kC * 256;      // q, k, v of a chunk: 48 KiB
constexpr int kOffV = 2 * kHalf;
constexpr int kOffT = 2 * kTileBytes;        // T: high and low tf32, each two atoms of 32 columns
constexpr int kTAtom = kC * 128;
constexpr int kPPart = kC * 128;             // P, two buffers of three bf16 pieces
constexpr int kPBytes = 3 * kPPart;
constexpr int kOffP = kOffT + 4 * kTAtom;
constexpr int kOffStage = kOffP + 2 * kPBytes;          // the workspace's blocks, two buffers
constexpr int kStageBytes = 2 * kPart * 4;
constexpr int kOffMeta = kOffStage + 2 * kStageBytes;

struct Gates {
  __align__(16) float gam[kC];               // gamma
  float tail[kC];                            // exp(cl_last - cl)
  float g;                                   // gamma of the last token
};
enum Bar {
  kFull0, kFull1,      // q / k / v of a chunk have landed
  kStage0, kStage1,    // T and P of a chunk have landed
  kTile0, kTile1,      // ... and are clean past the sequence's end
  kGates0, kGates1, kGates2, kGates3,       // gates of a chunk: a barrier per buffer
  kPrepared0, kPrepared1,                   // T and P of a chunk in place
  kSHigh, kS0, kS1,    // pieces of S: the high ones, the others of the first and second 16 columns
  kSK, kR, kTR,
  kU0, kU1, kU2,       // pieces of U~ (and, with the last, U for the output)
  kSQ, kD, kOFree,
  kO0, kO1,            // o of a chunk: its tile and operands are done with
  kEnd, kBars
};
struct Meta {
  unsigned long long bar[kBars];
  uint32_t tmem;
  Gates gate[4];
};
constexpr int kSmemBytes = kOffMeta + (int)sizeof(Meta) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

// Instruction descriptor bit: B is N-major (its N index contiguous in shared memory).
constexpr uint32_t kBTransposed = 1u << 16;
// Operand with N contiguous, 128-byte swizzle: groups of 64 N elements `lbo` bytes apart, groups
// of 8 K rows (of 128 bytes) `sbo` bytes apart.
__device__ __forceinline__ uint64_t desc_n_major(uint32_t start, uint32_t lbo, uint32_t sbo) {
  return ptx::smem_desc_sw128(start, sbo) & ~(0x3FFFull << 16) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
}

// Values into kN pieces, packed two to a column, at col, col + step, ...
template <int kN>
__device__ __forceinline__ void store_pieces(uint32_t col, uint32_t step, float (&x)[16]) {
#pragma unroll
  for (int p = 0; p < kN; ++p) {
    uint32_t packed[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) packed[i] = cut(x[2 * i], x[2 * i + 1]);
    tmem_store8(col + p * step, packed);
  }
}

// Waits and arrivals of one CTA.  A role whose wait runs out waits for nothing more: the chain and
// the warps that place T and P then go through their remaining barriers without effect on the
// outputs, so that none of them is left at one; the others stop.  (The code of a chunk is long, and
// waits are kept short: what a role's loop does not fit into the instruction cache it fetches anew.)
struct Sync {
  Meta *mt;
  __device__ __forceinline__ uint32_t at(int b) const { return ptx::smem_addr(&mt->bar[b]); }
  __device__ __forceinline__ bool wait(int b, int use) const {
    return ptx::mbar_wait_bounded(at(b), use & 1, kSpinLimit);
  }
  // one arrival per warp, after what its lanes wrote to tensor memory
  __device__ __forceinline__ void arrive_tmem(int b) const {
    ptx::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(at(b));
  }
  __device__ __forceinline__ void arrive_warp(int b) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(at(b));
  }
};
template <bool kGdn, typename Tout>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, SequenceArgs a) {
  extern __shared__ unsigned char smem_dyn[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Meta &mt = *reinterpret_cast<Meta *>(sm + kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.H, item = blockIdx.x, s = item / H, h = item % H, kh = qk_head(h, H, a.Hk);
  int lo, n;
  const bool in = sequence_range(a.offsets, s, a.T, a.max_len, lo, n);
  if (!__syncthreads_and(in && sequence_rises(a.offsets, s, lo, tid, kThreads))) {
    if (tid == 0) set_status(a.ws, TV_ERR_BAD_TREE, s);
    return;
  }
  const size_t state = (size_t)item * 128 * 128;
  if (n == 0) {
    for (int e = tid; e < 128 * 128 / 4; e += kThreads) {
      const float4 x = a.S_in ? reinterpret_cast<const float4 *>(a.S_in + state)[e]
                              : make_float4(0.f, 0.f, 0.f, 0.f);
      reinterpret_cast<float4 *>(a.S_out + state)[e] = x;
    }
    return;
  }
  const int chunks = (n + kC - 1) / kC;
  const uint32_t sbase = ptx::smem_addr(sm);
  const Sync sy{&mt};
  if (tid == 0) {
    for (int b = 0; b < kBars; ++b) {
      const int count = b == kTile0 || b == kTile1 || b == kPrepared0 || b == kPrepared1 ? kPrep
                        : (b >= kSHigh && b <= kS1) || b == kR || (b >= kU0 && b <= kU2) || b == kOFree ? kChain : 1;
      ptx::mbar_init(sy.at(b), count);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_addr(&mt.tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = 0;             // all 512 columns are this CTA's

  bool late = false;                   // a wait of this role has run out
  if (warp < kChain) {
    // ==== the chain ============================================================================
    const int part = warp >> 2, v = 32 * (warp & 3) + lane;      // columns 32 part, tokens 16 part
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float S[2][16];
    const size_t mine = state + (size_t)v * 128 + 32 * part;
    // (a first decay of zero starts afresh, also from NaN and infinity, which the products would spread)
    const bool from = a.S_in && expf(a.log_a[(size_t)lo * H + h]) != 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = from ? *reinterpret_cast<const float4 *>(a.S_in + mine + 4 * i)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i >> 2][4 * (i & 3)] = x.x;
      S[i >> 2][4 * (i & 3) + 1] = x.y;
      S[i >> 2][4 * (i & 3) + 2] = x.z;
      S[i >> 2][4 * (i & 3) + 3] = x.w;
    }
    Tout *out = static_cast<Tout *>(a.out);
    const size_t out_row = (size_t)H * 128;
    // 16 gates of this warp's tokens
    const auto gates = [&](const float *g, float (&x)[16]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 y = *reinterpret_cast<const float4 *>(g + 16 * part + 4 * j);
        x[4 * j] = y.x;
        x[4 * j + 1] = y.y;
        x[4 * j + 2] = y.z;
        x[4 * j + 3] = y.w;
      }
    };
    // o of chunk c, from tensor memory to its rows
    const auto write_out = [&](int c, bool valid) {
      float o[16], x[16], gam[16];
      gates(mt.gate[c & 3].gam, gam);
      tmem_load(tl + kColSQ + 16 * part, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= gam[j];
      tmem_load(tl + kColUP + 16 * part, o);
      sy.arrive_tmem(kOFree);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] += x[j];
      const int first = c * kC + 16 * part, rows = valid ? n - first : 0;
      Tout *p = out + (lo + first) * out_row + h * 128 + v;
      if (rows >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) put(p + j * out_row, o[j]);
      } else {
#pragma unroll 1
        for (int j = 0; j < rows; ++j, p += out_row) {
          float y = o[0];
#pragma unroll
          for (int i = 1; i < 16; ++i) y = i == j ? o[i] : y;
          put(p, y);
        }
      }
    };
    // this thread's 16 values of V of chunk c
    uint32_t vp[8];
    const auto fetch_v = [&](int c) {
      const bool there = sy.wait(kFull0 + (c & 1), c >> 1) && sy.wait(kTile0 + (c & 1), c >> 1);
      const uint16_t *vt =
          reinterpret_cast<const uint16_t *>(sm + (c & 1) * kTileBytes + kOffV) + 16 * part * 128 + v;
#pragma unroll
      for (int j = 0; j < 16; j += 2) vp[j / 2] = vt[j * 128] | (uint32_t)vt[(j + 1) * 128] << 16;
      return there;
    };
    bool ok = fetch_v(0);
    for (int c = 0; c < chunks; ++c) {
      const Gates &gt = mt.gate[c & 3];
      // S into its pieces, the high ones first: S K^T starts on them
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t packed[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          packed[i] = __byte_perm(__float_as_uint(S[g][2 * i]), __float_as_uint(S[g][2 * i + 1]), 0x7632);
        tmem_store8(tl + kColS + 16 * part + 8 * g, packed);
      }
      ptx::tmem_wait_st();
      sy.arrive_tmem(kSHigh);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = S[g][i] - __uint_as_float(__float_as_uint(S[g][i]) & 0xFFFF0000u);
        store_pieces<2>(tl + kColS + 64 + 16 * part + 8 * g, 64, x);
        ptx::tmem_wait_st();
        sy.arrive_tmem(kS0 + g);
      }
      // o of the chunk before: gated, while R T^T is computed; scalar decay, now, which frees what the
      // operands are written over (storing it after them: 111 us for 8 x 1000 tokens against 90)
      const auto write_last = [&] {
        if (c == 0) return;
        ok = ok && sy.wait(kO0 + ((c - 1) & 1), (c - 1) >> 1);
        ptx::tc_fence_after();
        write_out(c - 1, ok);
      };
      if (!kGdn) write_last();
      ok = ok && sy.wait(kGates0 + (c & 3), c >> 2);
      // V (scalar decay: U = V at once)
      float u[16], gate[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[2 * j] = __uint_as_float(vp[j] << 16);
        u[2 * j + 1] = __uint_as_float(vp[j] & 0xFFFF0000u);
      }
      if (kGdn) {
        gates(gt.gam, gate);
        ok = ok && sy.wait(kSK, c);
        ptx::tc_fence_after();
        {
          // R in two tf32 halves
          float r[16];
          tmem_load(tl + kColSK + 16 * part, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            u[j] = fmaf(-gate[j], r[j], u[j]);
            r[j] = tf32_round(u[j]);
            u[j] -= r[j];
          }
          ptx::tmem_st16(tl + kColR + 16 * part, r);
          ptx::tmem_st16(tl + kColR + 64 + 16 * part, u);
        }
        ptx::tmem_wait_st();
        sy.arrive_tmem(kR);
        write_last();
        gates(gt.tail, gate);
        ok = ok && sy.wait(kTR, c);
        ptx::tc_fence_after();
        tmem_load(tl + kColSK + 16 * part, u);
      } else {
        gates(gt.tail, gate);
      }
      // pieces of U~ (decayed to the chunk's end), one after the other, and U for the output
      {
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = u[j] * gate[j];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          uint32_t packed[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) packed[i] = cut(x[2 * i], x[2 * i + 1]);
          tmem_store8(tl + kColUt + 32 * p + 8 * part, packed);
          if (p < 2) {
            ptx::tmem_wait_st();
            sy.arrive_tmem(kU0 + p);
          }
        }
        uint32_t packed[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) packed[i] = cut(u[2 * i], u[2 * i + 1]);
        tmem_store8(tl + kColU + 8 * part, packed);
        store_pieces<2>(tl + kColSK + 16 * part, 8, u);      // over the accumulator it came from
      }
      ptx::tmem_wait_st();
      sy.arrive_tmem(kU2);
      if (c + 1 < chunks) ok = ok && fetch_v(c + 1);
      // S' = g S + D
      const float decay = gt.g;
      ok = ok && sy.wait(kD, c);
      ptx::tc_fence_after();
      {
        float d[32];
        tmem_load(tl + kColD + 32 * part, d);
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i >> 4][i & 15] = fmaf(decay, S[i >> 4][i & 15], d[i]);
      }
      ptx::tc_fence_before();
      group_sync(1, kChain * 32);              // D has been read: its columns take the pieces
      ptx::tc_fence_after();
    }
    ok = ok && sy.wait(kO0 + ((chunks - 1) & 1), (chunks - 1) >> 1);
    ptx::tc_fence_after();
    write_out(chunks - 1, ok);
    late = !ok;
    if (ok) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4 *>(a.S_out + mine + 4 * i) =
            make_float4(S[i >> 2][4 * (i & 3)], S[i >> 2][4 * (i & 3) + 1], S[i >> 2][4 * (i & 3) + 2],
                        S[i >> 2][4 * (i & 3) + 3]);
    }
  } else if (warp < kChain + kPrep) {
    // ==== T and P of every chunk into their operands ============================================
    const int pt = tid - kChain * 32;
    // blocks above the diagonal stay zero
    for (int e = pt; e < (4 * kTAtom + 2 * kPBytes) / 16; e += kPrep * 32)
      *reinterpret_cast<uint4 *>(sm + kOffT + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
    // what one of these warps zeroes, another may write: none starts before all are through
    group_sync(2, kPrep * 32);
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      unsigned char *tile = sm + (c & 1) * kTileBytes;
      ok = ok && sy.wait(kFull0 + (c & 1), c >> 1);
      const int rows = min(kC, n - c * kC);
      if (rows < kC) {
        for (int e = pt; e < (kC - rows) * 32; e += kPrep * 32) {
          const int r = rows + (e >> 5), x = e & 31;       // 16 chunks of a k row, 16 of a v row
          unsigned char *p = x < 16 ? tile + (x >> 3) * kHalf + kKRow + r * 128 + (x & 7) * 16
                                    : tile + kOffV + r * 256 + (x & 15) * 16;
          *reinterpret_cast<uint4 *>(p) = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
      }
      sy.arrive_warp(kTile0 + (c & 1));
      ok = ok && sy.wait(kStage0 + (c & 1), c >> 1);
      const float4 *blocks = reinterpret_cast<const float4 *>(sm + kOffStage + (c & 1) * kStageBytes);
      // (P's buffer was last read by chunk c - 2, before this chunk's tile came)
      unsigned char *po = sm + kOffP + (c & 1) * kPBytes;
      if (kGdn && c > 0) ok = ok && sy.wait(kTR, c - 1);              // T of the chunk before has been read
#pragma unroll
      for (int e0 = 0; e0 < kPart / 4; e0 += kPrep * 32) {
        const int e = e0 + pt, b = e >> 6, I = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3;
        const int row = 16 * I + (e >> 2 & 15), i4 = 4 * (b - I * (I + 1) / 2) + (e & 3);   // columns 4 i4
        const float4 x = blocks[e];
        float y[4] = {x.x, x.y, x.z, x.w};
        const int at = row * 128 + (((i4 >> 1) ^ (row & 7)) << 4) + (i4 & 1) * 8;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const uint32_t lo2 = cut(y[0], y[1]), hi2 = cut(y[2], y[3]);
          *reinterpret_cast<uint2 *>(po + p * kPPart + at) = make_uint2(lo2, hi2);
        }
        if (kGdn) {
          // T's blocks are transposed: four rows of column e / 4
          const float4 t = blocks[kPart / 4 + e];
          const float y[4] = {t.x, t.y, t.z, t.w};
          const int col = 16 * (b - I * (I + 1) / 2) + (e >> 2 & 15), row0 = 16 * I + 4 * (e & 3);
          unsigned char *to = sm + kOffT + (col >> 5) * kTAtom + row0 * 128 + (col & 3) * 4;
          const int chunk = ((col >> 2 & 7) ^ (row0 & 4)) << 4;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float hi = tf32_round(y[r]);
            float *at_r = reinterpret_cast<float *>(to + r * 128 + (chunk ^ (r << 4)));
            *at_r = hi;
            at_r[2 * kTAtom / 4] = y[r] - hi;
          }
        }
      }
      ptx::fence_proxy_async_smem();
      sy.arrive_warp(kPrepared0 + (c & 1));
    }
    late = !ok;
  } else if (warp == kChain + kPrep) {
    // ==== gates and copies ========================================================================
    const bool one = elect_one();
    if (one) {
      ptx::prefetch_tmap(&tm_q);
      ptx::prefetch_tmap(&tm_k);
      ptx::prefetch_tmap(&tm_v);
    }
    int loaded = 0, staged = 0;
    const auto load = [&](int c) {
      const uint32_t b = sbase + (c & 1) * kTileBytes, bar = sy.at(kFull0 + (c & 1));
      if (one) {
        ptx::mbar_arrive_expect_tx(bar, kTileBytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ptx::tma_load_3d(b + half * kHalf + kKRow, &tm_k, bar, half * 64, kh, lo + c * kC);
          ptx::tma_load_3d(b + half * kHalf, &tm_q, bar, half * 64, kh, lo + c * kC);
        }
        ptx::tma_load_3d(b + kOffV, &tm_v, bar, 0, h, lo + c * kC);
      }
      loaded = c + 1;
    };
    const auto stage = [&](int c) {
      constexpr uint32_t kBytes = slot_floats(kGdn) * 4;
      const uint32_t bar = sy.at(kStage0 + (c & 1));
      if (one) {
        ptx::mbar_arrive_expect_tx(bar, kBytes);
        ptx::bulk_load(sbase + kOffStage + (c & 1) * kStageBytes, slot_at(a, kGdn, lo / kC + s + c, h), kBytes, bar);
      }
      staged = c + 1;
    };
    float la[2];
    const auto fetch = [&](int c) {               // tokens 2 lane and 2 lane + 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = c * kC + 2 * lane + e;
        la[e] = t < n ? a.log_a[(size_t)(lo + t) * H + h] : 0.f;
      }
    };
    const auto gates = [&](int c) {
      Gates &gt = mt.gate[c & 3];
      const double x[2] = {log2_decay(la[0]), log2_decay(la[1])};
      if (c + 1 < chunks) fetch(c + 1);
      const double sum = prefix(x), all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const double cl = e ? sum : sum - x[1];
        gt.gam[2 * lane + e] = exp2f((float)cl);
        gt.tail[2 * lane + e] = exp2f((float)(all - cl));
      }
      if (lane == 31) gt.g = exp2f((float)all);
      sy.arrive_warp(kGates0 + (c & 3));
    };
    load(0);
    stage(0);
    if (chunks > 1) {
      load(1);
      stage(1);
    }
    fetch(0);
    gates(0);
    // iteration c: chunk c - 1 is over; chunk c + 1 needs the gates that follow, so the chunks
    // cannot run away from these waits
    bool ok = true;
    for (int c = 0; ok && c < chunks; ++c) {
      if (c > 0) {
        if (!(ok = sy.wait(kO0 + ((c - 1) & 1), (c - 1) >> 1))) break;
        if (c + 1 < chunks) load(c + 1);
      }
      if (c + 1 < chunks) gates(c + 1);
      if (c + 2 < chunks) {
        if (!(ok = sy.wait(kPrepared0 + (c & 1), c >> 1))) break;
        stage(c + 2);
      }
    }
    late = !ok;
    for (int c = loaded > 2 ? loaded - 2 : 0; c < loaded; ++c)
      ptx::mbar_wait_bounded(sy.at(kFull0 + (c & 1)), (c >> 1) & 1, kSpinLimit);
    for (int c = staged > 2 ? staged - 2 : 0; c < staged; ++c)
      ptx::mbar_wait_bounded(sy.at(kStage0 + (c & 1)), (c >> 1) & 1, kSpinLimit);
  } else {
    // ==== MMAs: the warp goes through the waits together, one lane issues ========================
    const bool one = elect_one();
    constexpr uint32_t kId64 = ptx::idesc_bf16_f32(128, 64), kId128 = ptx::idesc_bf16_f32(128, 128);
    constexpr uint32_t kIdT = ptx::idesc_tf32_f32(128, 64);
    constexpr uint32_t tm = 0;         // all 512 columns: the first one's address
    // descriptors of the operands at their first step; a step adds its offset in 16 bytes
    const uint64_t d_qk = ptx::smem_desc_sw128(sbase, 1024);
    const uint64_t d_kn = desc_n_major(sbase + kKRow, kHalf, 1024);
    const uint64_t d_t = ptx::smem_desc_sw128(sbase + kOffT, 1024);
    const uint64_t d_p = ptx::smem_desc_sw128(sbase + kOffP, 1024);
    // step kk of a K-major operand in columns of 128 bytes `half` bytes apart
    const auto step = [](int half, int kk) { return (uint64_t)(((kk >> 2) * half + (kk & 3) * 32) >> 4); };
    bool ok = true;
    for (int c = 0; ok && c < chunks; ++c) {
      const uint64_t q = d_qk + ((c & 1) * kTileBytes >> 4), k = q + (kKRow >> 4);
      // S in pieces; by then the chunk before is through with its tiles and its operands
      if (!(ok = sy.wait(kTile0 + (c & 1), c >> 1) && (c == 0 || sy.wait(kO0 + ((c - 1) & 1), (c - 1) >> 1)) &&
                 sy.wait(kSHigh, c)))
        break;
      ptx::tc_fence_after();
      if (kGdn) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16(one, tm + kColSK, tm + kColS + 8 * kk, k + step(kHalf, kk), kId64, kk > 0);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!(ok = ok && sy.wait(kS0 + g, c))) break;
        ptx::tc_fence_after();
        if (kGdn) {
#pragma unroll
          for (int kk = g; kk < 8; kk += 2)
#pragma unroll
            for (int p = 1; p < 3; ++p)
              mma_f16(one, tm + kColSK, tm + kColS + 64 * p + 8 * kk, k + step(kHalf, kk), kId64, 1);
        }
      }
      if (!ok) break;
      if (kGdn) mma_done(one, sy.at(kSK));
      if (!(ok = sy.wait(kPrepared0 + (c & 1), c >> 1))) break;
      if (kGdn) {
        if (!(ok = sy.wait(kR, c))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t hi = d_t + step(kTAtom, kk), low = hi + (2 * kTAtom >> 4);
          mma_tf32(one, tm + kColSK, tm + kColR + 8 * kk, hi, kIdT, kk > 0);
          mma_tf32(one, tm + kColSK, tm + kColR + 8 * kk, low, kIdT, 1);
          mma_tf32(one, tm + kColSK, tm + kColR + 64 + 8 * kk, hi, kIdT, 1);
        }
        mma_done(one, sy.at(kTR));
      }
      if (c > 0 && !(ok = sy.wait(kOFree, c - 1))) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int p = 0; p < 3; ++p)
          mma_f16(one, tm + kColSQ, tm + kColS + 64 * p + 8 * kk, q + step(kHalf, kk), kId64, kk + p > 0);
      mma_done(one, sy.at(kSQ));
      // U~ K over the columns of S, which S Q^T must have read
      if (!(ok = sy.wait(kSQ, c))) break;
      const uint64_t kn = d_kn + ((c & 1) * kTileBytes >> 4);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        if (!(ok = ok && sy.wait(kU0 + p, c))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16(one, tm + kColD, tm + kColUt + 32 * p + 8 * kk, kn + (kk * 2048 >> 4), kId128 | kBTransposed,
                  kk + p > 0);
      }
      if (!ok) break;
      mma_done(one, sy.at(kD));
      {
        const uint64_t pd = d_p + ((c & 1) * kPBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          // piece p of U at its columns, piece r of P
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const uint32_t up = p == 0 ? kColU + 8 * kk : kColSK + 16 * kk + 8 * (p - 1);
#pragma unroll
            for (int r = 0; r < 3 - p; ++r)
              mma_f16(one, tm + kColUP, tm + up, pd + ((r * kPPart + kk * 32) >> 4), kId64, kk + p + r > 0);
          }
        }
        mma_done(one, sy.at(kO0 + (c & 1)));
      }
    }
    late = !ok;
    // what was issued has to end before the CTA does
    if (one) ptx::mma_commit(sy.at(kEnd));
    ptx::mbar_wait_bounded(sy.at(kEnd), 0, kSpinLimit);
  }
  __syncwarp();
  ptx::tc_fence_before();
  const bool timed_out = __syncthreads_or(late);
  if (timed_out && tid == 0) set_status(a.ws, TV_ERR_TIMEOUT, s);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(mt.tmem, 512);
  }
}

template <bool kGdn, typename Tout>
cudaError_t launch(const SequenceArgs &a, cudaStream_t st) {
  CUtensorMap tq, tk, tv_;
  if (!make_node_map(&tq, a.q, a.Hk, a.T, kC) || !make_node_map(&tk, a.k, a.Hk, a.T, kC) ||
      !make_row_map(&tv_, const_cast<void *>(a.v), true, a.H, a.T, kC))
    return cudaErrorInvalidValue;
  auto kernel = prefill_tc_kernel<kGdn, Tout>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kernel<<<a.B * a.H, kThreads, kSmemBytes, st>>>(tq, tk, tv_, a);
  return cudaGetLastError();
}

}  // namespace

size_t prefill_tc_workspace(long long T, long long B, long long H, int mode) {
  return kWorkspaceBytes + slots(T, B) * H * slot_floats(mode == TV_MODE_GDN) * 4;
}

cudaError_t launch_prefill_tc(const SequenceArgs &a, int mode, int out_dtype, cudaStream_t st) {
  const cudaError_t e = launch_prefill_prepare(a, mode, st);
  if (e != cudaSuccess) return e;
  if (mode == TV_MODE_GDN)
    return out_dtype == TV_F32 ? launch<true, float>(a, st) : launch<true, __nv_bfloat16>(a, st);
  return out_dtype == TV_F32 ? launch<false, float>(a, st) : launch<false, __nv_bfloat16>(a, st);
}

}  // namespace tv
