// Whole prompts through the recurrence on tensor cores: bf16 q / k / v, dk = dv = 128, gated
// delta rule or scalar decay, fp32 states.
//
// A sequence is taken in chunks of 64 tokens.  With cl the sum of log_a inside the chunk,
// gamma = exp(cl), S the state before it and g = gamma of its last token, the recurrence's
// closed form is
//     R_n = b_n v_n - b_n gamma_n S k_n,    U = T R,  T = (I + L)^-1,
//     L[n][i] = b_n exp(cl_n - cl_i) k_n.k_i  (i < n),
//     o_n = gamma_n S q_n + sum_{i <= n} P[n][i] u_i,  P[n][i] = exp(cl_n - cl_i) q_n.k_i,
//     S' = g S + sum_i exp(cl_last - cl_i) u_i k_i^T          (scalar decay: U = V).
// Everything is kept transposed as in the verify kernels: tensor-memory lane = value row v.
//
// Precision.  States are fp32 and every product on their path is as good: a bf16 operand (k, q)
// meets an fp32 one cut into three bf16 pieces of 8 bits (exact), T and R meet as pairs of tf32
// (22 bits; the product of the two low parts, 2^-22 and less, is left out).  The output's own
// products are as good where out is fp32.  Where it is bf16 (2^-8), S Q^T takes two pieces of S
// (16 bits) and U P^T is one tf32 product (11 bits).  Decay ratios are powers of two of a
// difference of sums kept as an fp32 pair.
//
// One CTA of 13 warps per (sequence, head), one per SM.  The chain of a chunk is
//     S -> [S K^T] -> R -> [R T^T] -> U -> [U~ K] -> S'          ([..] tensor core),
// and everything else is done beside it:
//   warps 0-7   the chain: S in registers (lane v, 64 of 128 columns each), its pieces, R, U and
//               its pieces into tensor memory; gamma S q scaled, the previous chunk's o stored.
//   warps 8-11  the next chunk's gates, Gram blocks [Q;K] K^T, T (16 x 16 diagonal blocks by
//               substitution, the rest by block products) and P, into operand tiles.
//   warp 12     one lane issues the copies (TMA, two q / k / v buffers) and the MMAs:
//               S K^T, the next Gram block, R T^T, S Q^T, U~ K, U P^T.
// Tensor memory (512 columns): [0,192) the pieces of S, D = U~ K over [0,128); [192,256) S K^T,
// then U, then low pieces of U; [256,320) S Q^T, then o; [320,448) R as two tf32 halves, then the
// pieces of U~ and the high piece of U; [448,512) the Gram block.
// Rows of a last partial chunk past the sequence are zeroed in shared memory (k and v), so that
// they add nothing.
//
// Every wait is bounded: one that runs out records TV_ERR_TIMEOUT on the status word and ends the
// CTA after its copies and MMAs (bounded again).
#include "serving.cuh"
#include "tc_ptx.cuh"
#include "tmaps.cuh"

namespace tv {
namespace {

constexpr int kC = 64;                       // tokens per chunk
constexpr int kChain = 8;                    // chain warps
constexpr int kPrep = 4;                     // preparing warps
constexpr int kThreads = (kChain + kPrep + 1) * 32;
constexpr uint32_t kSpinLimit = 1u << 22;

// tensor memory columns
constexpr uint32_t kColS = 0, kColD = 0, kColSK = 192, kColO = 256, kColR = 320, kColG = 448;
constexpr uint32_t kColUt = 320, kColU = 416;

// dynamic shared memory, from a 1024-byte aligned base
constexpr int kHalf = 2 * kC * 128;          // 64 columns of [Q ; K]: 128 rows of 128 bytes
constexpr int kKRow = kC * 128;              // K rows inside a half
constexpr int kVHalf = kC * 128;
constexpr int kTileBytes = 2 * kHalf + 2 * kVHalf;      // q, k, v of a chunk: 48 KiB
constexpr int kOffV = 2 * kHalf;
constexpr int kOffT = 2 * kTileBytes;        // T: high and low tf32, each two atoms of 32 columns
constexpr int kTAtom = kC * 128;
constexpr int kPPart = kC * 128;             // P, two buffers: three bf16 pieces, or two tf32 atoms
constexpr int kPBytes = 3 * kPPart;
constexpr int kOffP = kOffT + 4 * kTAtom;
constexpr int kOffMeta = kOffP + 2 * kPBytes;
constexpr int kLd = 68;                      // row of the fp32 work matrices

struct Gates {
  __align__(16) float clh[kC];               // cl in powers of two, as a pair
  float cll[kC];
  float end[kC];                             // exp(cl at the end of the block of 16 - cl)
  float gam[kC], bg[kC], bq[kC], tail[kC];   // gamma, b gamma, b, exp(cl_last - cl)
  float g;                                   // gamma of the last token
};
enum Bar {
  kFull0, kFull1,      // q / k / v of a chunk have landed
  kTile,               // ... and are clean past the sequence's end
  kGates0, kGates1,    // gates of a chunk (two barriers: the preparing warps run ahead)
  kGram, kGramFree,    // Gram block computed / read
  kPrepared,           // T and P of a chunk in place
  kS, kSK, kR, kTR, kU, kSQ, kScaled, kD, kO, kOFree, kEnd, kBars
};
struct Meta {
  unsigned long long bar[kBars];
  uint32_t tmem;
  int fail;
  __align__(16) float L[kC][kLd];
  __align__(16) float T[kC][kLd];
  float X[4][16][20];                        // scratch of the preparing warps
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

// 32 columns of a warp's 32 lanes, complete on return.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&r)[32]) {
  uint32_t u[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
        "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}

// Two values cut: the packed upper halves (a bf16 piece each), leaving what is left of the values.
// Three pieces hold a value exactly.
__device__ __forceinline__ uint32_t cut(float &x0, float &x1) {
  const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
  const uint32_t na = (a & 0xFFFF0000u) ^ 0x80000000u, nb = (b & 0xFFFF0000u) ^ 0x80000000u;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "r"(na), "r"(nb));
  return __byte_perm(a, b, 0x7632);
}
// 32 values into kN pieces of 16 columns each, at col, col + step, ...
template <int kN>
__device__ __forceinline__ void store_pieces(uint32_t col, uint32_t step, float (&x)[32]) {
#pragma unroll
  for (int p = 0; p < kN; ++p) {
    float packed[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) packed[i] = __uint_as_float(cut(x[2 * i], x[2 * i + 1]));
    ptx::tmem_st16(col + p * step, packed);
  }
}
__device__ __forceinline__ float tf32_round(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xFFFFE000u);
}
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void put(float *p, float x) { __stcs(p, x); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Waits and arrivals of one CTA.  A wait that runs out is recorded once; from then on no wait
// waits.  The chain and preparing warps then go through their remaining barriers without effect
// on the outputs, so that none of them is left at a barrier; the issuing thread stops.
struct Sync {
  Meta *mt;
  int *ws;
  int item;
  __device__ __forceinline__ uint32_t at(int b) const { return ptx::smem_addr(&mt->bar[b]); }
  __device__ __forceinline__ bool wait(int b, int use) const {
    const uint32_t a = at(b), parity = use & 1;
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
      if (ptx::mbar_try_wait(a, parity)) return true;
      if ((i & 15) == 0 && *reinterpret_cast<volatile int *>(&mt->fail)) return false;
    }
    *reinterpret_cast<volatile int *>(&mt->fail) = 1;
    set_status(ws, TV_ERR_TIMEOUT, item);
    return false;
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
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float both(uint64_t a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
  return x + y;
}

// acc[r] += row row0 + r of A times column `col` of B for 16 x 16 blocks: even and odd products in
// the halves of a packed pair.
template <int R>
__device__ __forceinline__ void block_product(uint64_t (&acc)[R], const float *A, int row0, const float *B,
                                              int ldb, int col) {
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const uint64_t b0 = pair(B[k * ldb + col], B[(k + 1) * ldb + col]);
    const uint64_t b1 = pair(B[(k + 2) * ldb + col], B[(k + 3) * ldb + col]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 a = *reinterpret_cast<const float4 *>(A + (row0 + r) * kLd + k);
      acc[r] = fma2(pair(a.x, a.y), b0, fma2(pair(a.z, a.w), b1, acc[r]));
    }
  }
}

// T[row][i] into the operand tiles (high and low tf32).
__device__ __forceinline__ void put_t(unsigned char *sm, int row, int i, float t) {
  const int at = kOffT + (i >> 5) * kTAtom + row * 128 + ((((i >> 2) & 7) ^ (row & 7)) << 4) + (i & 3) * 4;
  const float hi = tf32_round(t);
  *reinterpret_cast<float *>(sm + at) = hi;
  *reinterpret_cast<float *>(sm + at + 2 * kTAtom) = t - hi;
}

// Blocks (J + 1 .. 3, J) of T, a warp's kCols columns of them: T_iJ = -T_ii sum_k L_ik T_kJ.  Columns
// of blocks do not depend on one another once the diagonal is there.
template <int kCols>
__device__ __forceinline__ void solve_columns(Meta &mt, unsigned char *sm, int J, int col0, int lane,
                                              float (*X)[20]) {
  constexpr int R = kCols / 2;                   // 32 / kCols groups of lanes share 16 rows
  const int col = col0 + (lane & (kCols - 1)), row = (lane / kCols) * R;
  for (int i = J + 1; i < 4; ++i) {
    uint64_t acc[R] = {};
    for (int k = J; k < i; ++k)
      block_product<R>(acc, &mt.L[16 * i][16 * k], row, &mt.T[16 * k][16 * J], kLd, col);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) X[row + r][col] = both(acc[r]);
    __syncwarp();
    uint64_t out[R] = {};
    block_product<R>(out, &mt.T[16 * i][16 * i], row, &X[0][0], 20, col);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float t = -both(out[r]);
      if (i < 3) mt.T[16 * i + row + r][16 * J + col] = t;
      put_t(sm, 16 * i + row + r, 16 * J + col, t);
    }
    __syncwarp();
  }
}

// T = (I + L)^-1 for the unit lower triangular system in mt.L, into the operand tiles, by the
// preparing warps: the four diagonal blocks by substitution, then two warps take the first column
// of blocks (nine products of 16 x 16 blocks in all), one the second (five), one the third (two).
__device__ __forceinline__ void invert(Meta &mt, unsigned char *sm, int aw, int lane) {
  {
    const int col = lane & 15, half = lane >> 4;
    float x[16];
    const float *D = &mt.L[16 * aw][16 * aw];
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
    // both halves hold the column: each writes every other row
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      const int row = 16 * aw + n + half, i = 16 * aw + col;
      const float t = half ? x[n + 1] : x[n];
      mt.T[row][i] = t;
      put_t(sm, row, i, t);
    }
  }
  group_sync(2, kPrep * 32);
  if (aw < 2) solve_columns<8>(mt, sm, 0, 8 * aw, lane, mt.X[aw]);
  else solve_columns<16>(mt, sm, aw - 1, 0, lane, mt.X[aw]);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <bool kGdn, typename Tout>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, SequenceArgs a) {
  constexpr int kNO = sizeof(Tout) == 2 ? 2 : 3;            // pieces in the output's products
  extern __shared__ unsigned char smem_dyn[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Meta &mt = *reinterpret_cast<Meta *>(sm + kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.H, item = blockIdx.x, s = item / H, h = item % H, kh = qk_head(h, H, a.Hk);
  int lo, n;
  if (!sequence_range(a.offsets, s, a.T, a.max_len, lo, n)) {
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
  const Sync sy{&mt, a.ws, s};
  if (tid == 0) {
    for (int b = 0; b < kBars; ++b) {
      const int count = b == kTile || b == kGramFree || b == kPrepared ? kPrep
                        : b == kS || b == kR || b == kU || b == kScaled || b == kOFree ? kChain : 1;
      ptx::mbar_init(sy.at(b), count);
    }
    ptx::fence_mbar_init();
    mt.fail = 0;
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_addr(&mt.tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = mt.tmem;

  if (warp < kChain) {
    // ==== the chain ============================================================================
    const int hf = warp >> 2, v = 32 * (warp & 3) + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float S[2][32];
    const size_t mine = state + (size_t)v * 128 + 64 * hf;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float4 x = a.S_in ? *reinterpret_cast<const float4 *>(a.S_in + mine + 4 * i)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i >> 3][4 * (i & 7)] = x.x;
      S[i >> 3][4 * (i & 7) + 1] = x.y;
      S[i >> 3][4 * (i & 7) + 2] = x.z;
      S[i >> 3][4 * (i & 7) + 3] = x.w;
    }
    Tout *out = static_cast<Tout *>(a.out);
    // o of chunk c, from tensor memory to its rows
    const auto write_out = [&](int c, bool valid) {
      float o[32];
      tmem_load32(tl + kColO + 32 * hf, o);
      sy.arrive_tmem(kOFree);
      const int first = c * kC + 32 * hf, rows = valid ? min(32, n - first) : 0;
      Tout *p = out + ((size_t)(lo + first) * H + h) * 128 + v;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < rows) put(p + (size_t)j * H * 128, o[j]);
    };
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const Gates &gt = mt.gate[c & 3];
      // S into its pieces
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = S[g][i];
        store_pieces<3>(tl + kColS + 32 * hf + 16 * g, 64, x);
      }
      ptx::tmem_wait_st();
      sy.arrive_tmem(kS);
      if (c > 0) {
        ok &= sy.wait(kO, c - 1);
        ptx::tc_fence_after();
        write_out(c - 1, ok);
      }
      // R (scalar decay: U = V at once)
      ok &= sy.wait(kGates0 + (c & 1), c >> 1);
      ok &= sy.wait(kFull0 + (c & 1), c >> 1);
      const unsigned char *vt = sm + (c & 1) * kTileBytes + kOffV + (v >> 6) * kVHalf + (v & 7) * 2;
      const int vc = (v & 63) >> 3;
      const auto value = [&](int i) {
        return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
            vt + i * 128 + ((vc ^ (i & 7)) << 4)));
      };
      float u[32];
      if (kGdn) {
        ok &= sy.wait(kSK, c);
        ptx::tc_fence_after();
        tmem_load32(tl + kColSK + 32 * hf, u);
        float low[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float high[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int i = 32 * hf + 16 * g + j;
            const float r = fmaf(-gt.bg[i], u[16 * g + j], gt.bq[i] * value(i));
            high[j] = tf32_round(r);
            low[j] = r - high[j];
          }
          ptx::tmem_st16(tl + kColR + 32 * hf + 16 * g, high);
          ptx::tmem_st16(tl + kColR + 64 + 32 * hf + 16 * g, low);
        }
        ptx::tmem_wait_st();
        sy.arrive_tmem(kR);
        ok &= sy.wait(kTR, c);
        ptx::tc_fence_after();
        tmem_load32(tl + kColSK + 32 * hf, u);
      } else {
        // (the operands of the chunk before have been read: its o has been written)
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = value(32 * hf + j);
      }
      // pieces of U~ (decayed to the chunk's end), and U for the output
      {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = u[j] * gt.tail[32 * hf + j];
        store_pieces<3>(tl + kColUt + 16 * hf, 32, x);
        if (kNO == 3) {
          float packed[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) packed[i] = __uint_as_float(cut(u[2 * i], u[2 * i + 1]));
          ptx::tmem_st16(tl + kColU + 16 * hf, packed);
          store_pieces<2>(tl + kColSK + 32 * hf, 16, u);
        } else {
          // U in tf32, over the accumulator it came from
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = tf32_round(u[16 * g + j]);
            ptx::tmem_st16(tl + kColSK + 32 * hf + 16 * g, y);
          }
        }
      }
      ptx::tmem_wait_st();
      sy.arrive_tmem(kU);
      // gamma S q
      ok &= sy.wait(kSQ, c);
      ptx::tc_fence_after();
      {
        float o[32];
        tmem_load32(tl + kColO + 32 * hf, o);
        float y[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = o[16 * g + j] * gt.gam[32 * hf + 16 * g + j];
          ptx::tmem_st16(tl + kColO + 32 * hf + 16 * g, y);
        }
        ptx::tmem_wait_st();
        sy.arrive_tmem(kScaled);
      }
      // S' = g S + D
      ok &= sy.wait(kD, c);
      ptx::tc_fence_after();
      const float decay = gt.g;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float d[32];
        tmem_load32(tl + kColD + 64 * hf + 32 * g, d);
#pragma unroll
        for (int i = 0; i < 32; ++i) S[g][i] = fmaf(decay, S[g][i], d[i]);
      }
      ptx::tc_fence_before();
      group_sync(1, kChain * 32);              // D has been read: its columns take the pieces
      ptx::tc_fence_after();
    }
    ok &= sy.wait(kO, chunks - 1);
    ptx::tc_fence_after();
    write_out(chunks - 1, ok);
    if (ok) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4 *>(a.S_out + mine + 4 * i) =
            make_float4(S[i >> 3][4 * (i & 7)], S[i >> 3][4 * (i & 7) + 1], S[i >> 3][4 * (i & 7) + 2],
                        S[i >> 3][4 * (i & 7) + 3]);
    }
  } else if (warp < kChain + kPrep) {
    // ==== gates, T and P of every chunk ==========================================================
    const int aw = warp - kChain;
    const uint32_t tl = tmem + ((uint32_t)(32 * aw) << 16);
    const int row = (32 * aw + lane) & 63;        // warps 0, 1: q rows; 2, 3: k rows
    float la[2] = {0.f, 0.f}, bb[2] = {0.f, 0.f};
    const auto fetch = [&](int c) {               // warp 0: tokens 2 lane and 2 lane + 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = c * kC + 2 * lane + e;
        const size_t at = (size_t)(lo + t) * H + h;
        la[e] = t < n ? a.log_a[at] : 0.f;
        bb[e] = kGdn && t < n ? a.b[at] : 0.f;
      }
    };
    if (aw == 0) fetch(0);
    // blocks above the diagonal of T stay zero
    for (int e = aw * 32 + lane; e < 4 * kTAtom / 16; e += kPrep * 32)
      *reinterpret_cast<uint4 *>(sm + kOffT + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
    group_sync(2, kPrep * 32);
    for (int c = 0; c < chunks; ++c) {
      Gates &gt = mt.gate[c & 3];
      unsigned char *tile = sm + (c & 1) * kTileBytes;
      sy.wait(kFull0 + (c & 1), c >> 1);
      const int rows = min(kC, n - c * kC);
      if (rows < kC) {
        for (int e = aw * 32 + lane; e < (kC - rows) * 32; e += kPrep * 32) {
          const int r = rows + (e >> 5), x = e & 31;       // 16 chunks of a k row, 16 of a v row
          unsigned char *p = x < 16 ? tile + (x >> 3) * kHalf + kKRow : tile + kOffV + (x >> 3 & 1) * kVHalf;
          *reinterpret_cast<uint4 *>(p + r * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
      }
      sy.arrive_warp(kTile);
      if (aw == 0) {
        // prefix sums in 64 bits: a decay of nearly zero spoils no later difference
        double x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = 1.4426950408889634 * (double)(la[e] < -1000.f ? -1000.f : la[e]);
        double sum = x[0] + x[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        const double all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const double cl = e ? sum : sum - x[1];
          const float hi = (float)cl;
          const int i = 2 * lane + e;
          const float gam = exp2f(hi);
          gt.clh[i] = hi;
          gt.cll[i] = (float)(cl - (double)hi);
          gt.gam[i] = gam;
          gt.bg[i] = bb[e] * gam;
          gt.bq[i] = bb[e];
          gt.tail[i] = exp2f((float)(all - cl));
          const double end = __shfl_sync(0xffffffffu, sum, lane | 7);
          gt.end[i] = exp2f((float)(end - cl));
        }
        if (lane == 31) gt.g = exp2f((float)all);
        sy.arrive_warp(kGates0 + (c & 1));
        if (c + 1 < chunks) fetch(c + 1);
      }
      group_sync(2, kPrep * 32);
      sy.wait(kGram, c);
      ptx::tc_fence_after();
      // rows of P (kept in registers) and of L
      float x[64];
      {
        float g0[32];
        tmem_load32(tl + kColG, g0);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = g0[i];
        tmem_load32(tl + kColG + 32, g0);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[32 + i] = g0[i];
      }
      sy.arrive_tmem(kGramFree);
      // decay ratios: inside a diagonal block of 16 one by one; before it as the product of
      // exp(cl_row - cl at the end of the column's block) and gate `end` of the column (both at
      // most 1 for decays)
      const float clh = gt.clh[row], cll = gt.cll[row];
      const bool is_k = aw >= 2;
      const float scale = is_k ? gt.bq[row] : 1.f;
      const int last = is_k ? row - 1 : row;
#pragma unroll
      for (int J = 0; J < 4; ++J) {
        const float before = scale * pow2((clh - gt.clh[16 * J + 15]) + (cll - gt.cll[16 * J + 15]));
        const bool diagonal = J >> 1 == (aw & 1);        // of some of the warp's rows
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int i = 16 * J + j;
          const float4 end = *reinterpret_cast<const float4 *>(&gt.end[i]);
          float f[4] = {before * end.x, before * end.y, before * end.z, before * end.w};
          if (diagonal) {
            const float4 ch = *reinterpret_cast<const float4 *>(&gt.clh[i]);
            const float4 cl = *reinterpret_cast<const float4 *>(&gt.cll[i]);
            const float d[4] = {(clh - ch.x) + (cll - cl.x), (clh - ch.y) + (cll - cl.y),
                                (clh - ch.z) + (cll - cl.z), (clh - ch.w) + (cll - cl.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (J == row >> 4) f[e] = scale * pow2(d[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i + e] = i + e <= last ? f[e] * x[i + e] : 0.f;
        }
      }
      if (!is_k) {
        // P into its operand (the buffer's last reader was chunk c - 2, before this chunk's tile)
        unsigned char *pt = sm + kOffP + (c & 1) * kPBytes + row * 128;
        if (kNO == 3) {
#pragma unroll
          for (int p = 0; p < 3; ++p) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint4 w;
              w.x = cut(x[8 * j], x[8 * j + 1]);
              w.y = cut(x[8 * j + 2], x[8 * j + 3]);
              w.z = cut(x[8 * j + 4], x[8 * j + 5]);
              w.w = cut(x[8 * j + 6], x[8 * j + 7]);
              *reinterpret_cast<uint4 *>(pt + p * kPPart + ((j ^ (row & 7)) << 4)) = w;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            *reinterpret_cast<float4 *>(pt + (j >> 3) * kPPart + (((j & 7) ^ (row & 7)) << 4)) =
                make_float4(tf32_round(x[4 * j]), tf32_round(x[4 * j + 1]), tf32_round(x[4 * j + 2]),
                            tf32_round(x[4 * j + 3]));
        }
      } else if (kGdn) {
#pragma unroll
        for (int i = 0; i < 64; i += 4)
          *reinterpret_cast<float4 *>(&mt.L[row][i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
      if (kGdn) {
        group_sync(2, kPrep * 32);
        if (c > 0) sy.wait(kTR, c - 1);            // T of the chunk before has been read
        invert(mt, sm, aw, lane);
      }
      ptx::fence_proxy_async_smem();
      sy.arrive_warp(kPrepared);
    }
  } else {
    // ==== copies and MMAs: the warp goes through the waits together, one lane issues ============
    const bool one = elect_one();
    if (one) {
      ptx::prefetch_tmap(&tm_q);
      ptx::prefetch_tmap(&tm_k);
      ptx::prefetch_tmap(&tm_v);
    }
    int loaded = 0;
    const auto load = [&](int c) {
      const uint32_t b = sbase + (c & 1) * kTileBytes, bar = sy.at(kFull0 + (c & 1));
      if (one) {
        ptx::mbar_arrive_expect_tx(bar, kTileBytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ptx::tma_load_3d(b + half * kHalf + kKRow, &tm_k, bar, half * 64, kh, lo + c * kC);
          ptx::tma_load_3d(b + half * kHalf, &tm_q, bar, half * 64, kh, lo + c * kC);
          ptx::tma_load_3d(b + kOffV + half * kVHalf, &tm_v, bar, half * 64, h, lo + c * kC);
        }
      }
      loaded = c + 1;
    };
    constexpr uint32_t kId64 = ptx::idesc_bf16_f32(128, 64), kId128 = ptx::idesc_bf16_f32(128, 128);
    constexpr uint32_t kIdT = ptx::idesc_tf32_f32(128, 64);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    // descriptors of the operands at their first step; a step adds its offset in 16 bytes
    const uint64_t d_qk = ptx::smem_desc_sw128(sbase, 1024);
    const uint64_t d_kn = desc_n_major(sbase + kKRow, kHalf, 1024);
    const uint64_t d_t = ptx::smem_desc_sw128(sbase + kOffT, 1024);
    const uint64_t d_p = ptx::smem_desc_sw128(sbase + kOffP, 1024);
    // step kk of a K-major operand in columns of 128 bytes `half` bytes apart
    const auto step = [](int half, int kk) { return (uint64_t)(((kk >> 2) * half + (kk & 3) * 32) >> 4); };
    const auto gram = [&](int c) {
      const uint64_t q = d_qk + ((c & 1) * kTileBytes >> 4), k = q + (kKRow >> 4);
      if (one) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16(tm + kColG, q + step(kHalf, kk), k + step(kHalf, kk), kId64, kk > 0);
        ptx::mma_commit(sy.at(kGram));
      }
    };
    bool ok = true;
    load(0);
    if (chunks > 1) load(1);
    if ((ok = sy.wait(kTile, 0))) gram(0);
    for (int c = 0; ok && c < chunks; ++c) {
      const uint64_t q = d_qk + ((c & 1) * kTileBytes >> 4), k = q + (kKRow >> 4);
      // S in pieces; by then the chunk before is through with its tiles and its operands
      if (!(ok = sy.wait(kS, c) && (c == 0 || sy.wait(kO, c - 1)))) break;
      ptx::tc_fence_after();
      if (kGdn && one) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int p = 0; p < 3; ++p)
            ptx::mma_bf16_tmem_a(tm + kColSK, tm + kColS + 64 * p + 8 * kk, k + step(kHalf, kk), kId64,
                                 kk + p > 0);
        ptx::mma_commit(sy.at(kSK));
      }
      if (c > 0 && c + 1 < chunks) load(c + 1);
      if (c + 1 < chunks) {
        if (!(ok = sy.wait(kTile, c + 1) && sy.wait(kGramFree, c))) break;
        ptx::tc_fence_after();
        gram(c + 1);
      }
      if (!(ok = sy.wait(kPrepared, c))) break;
      if (kGdn) {
        if (!(ok = sy.wait(kR, c))) break;
        ptx::tc_fence_after();
        if (one) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t hi = d_t + step(kTAtom, kk), low = hi + (2 * kTAtom >> 4);
            ptx::mma_tf32_tmem_a(tm + kColSK, tm + kColR + 8 * kk, hi, kIdT, kk > 0);
            ptx::mma_tf32_tmem_a(tm + kColSK, tm + kColR + 8 * kk, low, kIdT, 1);
            ptx::mma_tf32_tmem_a(tm + kColSK, tm + kColR + 64 + 8 * kk, hi, kIdT, 1);
          }
          ptx::mma_commit(sy.at(kTR));
        }
      }
      if (c > 0 && !(ok = sy.wait(kOFree, c - 1))) break;
      ptx::tc_fence_after();
      if (one) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int p = 0; p < kNO; ++p)
            ptx::mma_bf16_tmem_a(tm + kColO, tm + kColS + 64 * p + 8 * kk, q + step(kHalf, kk), kId64,
                                 kk + p > 0);
        ptx::mma_commit(sy.at(kSQ));
      }
      // U~ K over the columns of S, which S Q^T must have read
      if (!(ok = sy.wait(kU, c) && sy.wait(kSQ, c))) break;
      ptx::tc_fence_after();
      if (one) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t kd = d_kn + ((c & 1) * kTileBytes >> 4) + (kk * 2048 >> 4);
#pragma unroll
          for (int p = 0; p < 3; ++p)
            ptx::mma_bf16_tmem_a(tm + kColD, tm + kColUt + 32 * p + 8 * kk, kd, kId128 | kBTransposed,
                                 kk + p > 0);
        }
        ptx::mma_commit(sy.at(kD));
      }
      if (!(ok = sy.wait(kScaled, c))) break;
      ptx::tc_fence_after();
      if (one) {
        const uint64_t pd = d_p + ((c & 1) * kPBytes >> 4);
        if (kNO == 3) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // piece p of U at its columns, piece r of P
#pragma unroll
            for (int p = 0; p < 3; ++p) {
              const uint32_t up =
                  p == 0 ? kColU + 8 * kk : kColSK + 32 * (kk >> 1) + 16 * (p - 1) + 8 * (kk & 1);
#pragma unroll
              for (int r = 0; r < 3 - p; ++r)
                ptx::mma_bf16_tmem_a(tm + kColO, tm + up, pd + ((r * kPPart + kk * 32) >> 4), kId64, 1);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_tf32_tmem_a(tm + kColO, tm + kColSK + 8 * kk, pd + step(kPPart, kk), kIdT, 1);
        }
        ptx::mma_commit(sy.at(kO));
      }
    }
    // what was issued has to end before the CTA does
    if (one) ptx::mma_commit(sy.at(kEnd));
    ptx::mbar_wait_bounded(sy.at(kEnd), 0, kSpinLimit);
    for (int c = loaded > 2 ? loaded - 2 : 0; c < loaded; ++c)
      ptx::mbar_wait_bounded(sy.at(kFull0 + (c & 1)), (c >> 1) & 1, kSpinLimit);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <bool kGdn, typename Tout>
cudaError_t launch(const SequenceArgs &a, cudaStream_t st) {
  CUtensorMap tq, tk, tv_;
  if (!make_node_map(&tq, a.q, a.Hk, a.T, kC) || !make_node_map(&tk, a.k, a.Hk, a.T, kC) ||
      !make_node_map(&tv_, a.v, a.H, a.T, kC))
    return cudaErrorInvalidValue;
  auto kernel = prefill_tc_kernel<kGdn, Tout>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kernel<<<a.B * a.H, kThreads, kSmemBytes, st>>>(tq, tk, tv_, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_tc(const SequenceArgs &a, int mode, int out_dtype, cudaStream_t st) {
  if (mode == TV_MODE_GDN)
    return out_dtype == TV_F32 ? launch<true, float>(a, st) : launch<true, __nv_bfloat16>(a, st);
  return out_dtype == TV_F32 ? launch<false, float>(a, st) : launch<false, __nv_bfloat16>(a, st);
}

}  // namespace tv
