// What the two kernels of the tensor-core prefill share: chunks, the workspace's layout, operand
// pieces, tensor-memory access.  Included by those translation units only.
#pragma once

#include "serving.cuh"
#include "tc_ptx.cuh"
#include "tmaps.cuh"

namespace tv {
namespace prefill {

constexpr int kC = 64;                       // tokens per chunk

// Workspace behind the status word: a slot per chunk and head.  Chunk c of sequence s has slot
// offsets[s] / 64 + s + c, so sequences never meet.  A slot holds the blocks of 16 x 16 on and below
// the diagonal, block (i, j) at i (i + 1) / 2 + j, 16 floats to a row: those of P, then (gated delta
// rule) those of T, each transposed.
constexpr int kBlocks = 10;
constexpr int kPart = kBlocks * 256;         // floats of P or T
__host__ __device__ constexpr size_t slot_floats(bool gdn) { return (gdn ? 2 : 1) * kPart; }
__host__ __device__ constexpr long long slots(long long T, long long B) { return T / kC + B; }
__device__ __forceinline__ float *slot_at(const SequenceArgs &a, bool gdn, int slot, int h) {
  return reinterpret_cast<float *>(a.ws) + kWorkspaceBytes / 4 + ((size_t)slot * a.H + h) * slot_floats(gdn);
}

// A chunk of [Q ; K] in shared memory: two halves of 64 columns, 128 rows of 128 bytes each.
constexpr int kHalf = 2 * kC * 128;
constexpr int kKRow = kC * 128;              // K rows inside a half

// 16 or 32 columns of a warp's 32 lanes, complete on return.
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[16]) {
  uint32_t u[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[32]) {
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
// 8 columns from registers.
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Two values cut: the packed upper halves (a bf16 piece each), leaving what is left of the values.
// Three pieces hold a value exactly.
__device__ __forceinline__ uint32_t cut(float &x0, float &x1) {
  const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
  x0 -= __uint_as_float(a & 0xFFFF0000u);
  x1 -= __uint_as_float(b & 0xFFFF0000u);
  return __byte_perm(a, b, 0x7632);
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

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// log_a of a token, bounded: exp(-1000) is zero.
__device__ __forceinline__ double log2_decay(float la) {
  return 1.4426950408889634 * (double)(la < -1000.f ? -1000.f : la);
}
// Prefix sums over a chunk, two tokens to a lane, in 64 bits: a decay of nearly zero spoils no later
// difference.  x[e]: of token 2 lane + e; returns the sum up to token 2 lane + 1.
__device__ __forceinline__ double prefix(const double (&x)[2]) {
  double sum = x[0] + x[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, sum, o);
    if ((int)(threadIdx.x & 31) >= o) sum += y;
  }
  return sum;
}

// The issuing warp goes through its MMAs converged, one lane's `one` set: with no branch around
// them their operands stay in uniform registers (branched, an MMA took 50 to 70 cycles to issue).
__device__ __forceinline__ void mma_f16(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_tf32(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_done(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

}  // namespace prefill
}  // namespace tv
