// lod_pool_tc.cuh -- helpers of the block pool's tensor-core kernels.
#pragma once

#include <atomic>

#include "lod_pool.cuh"
#include "lod_tc.cuh"

namespace lod {
namespace {

constexpr int kKT = 128;               // keys of a tile
constexpr int kHalfBytes = 128 * 128;  // 128 rows x 64 bf16 channels

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void tma_load_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint32_t sw_off(int row, int chunk16) {  // 16-byte chunk of a 128B-swizzled row
  return (uint32_t)(row * 128 + (((chunk16 & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// ---------------------------------------------------------------- e4m3 -> bf16

// Four e4m3 codes as four bf16 (two words), each times 2^(E - 127).  Shifted
// into a bf16's exponent and mantissa, a code's low seven bits read as the
// code's value times 2^-120 (bias 127 against 7; a subnormal code becomes a
// subnormal bf16), so one product by 2^120 2^(E - 127) gives the row's value
// exactly.  f1 and f2 are that factor in two parts, as it can leave bf16's range.
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t f1, uint32_t f2, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  const uint32_t x = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u);
  const uint32_t y = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
  lo = hmul2_bf16(hmul2_bf16(x, f1), f2);
  hi = hmul2_bf16(hmul2_bf16(y, f1), f2);
}
// The same with one factor.
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t f, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  lo = hmul2_bf16(((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), f);
  hi = hmul2_bf16(((b >> 4) & 0x07f007f0u) | (b & 0x80008000u), f);
}
// The two factors of exponent byte E, each in both halves of a word.
__device__ __forceinline__ void e4m3_factors(int E, uint32_t& f1, uint32_t& f2) {
  // 2^(120 + e) = 2^(120 + min(e, 7)) * 2^(e - min(e, 7)); E = 255: NaN.  The
  // pool never holds e below -120; smaller ones read as 2^-120.
  int e = E - 127;
  e = e < -120 ? -120 : e;
  const int e1 = e < 7 ? e : 7;
  const uint32_t a = (uint32_t)(e1 + 120 + 127) << 7, b = E == 255 ? 0x7fc0u : (uint32_t)(e - e1 + 127) << 7;
  f1 = a | (a << 16);
  f2 = b | (b << 16);
}

// The register split (setmaxnreg) draws on what the CTA was launched with: a
// build whose kernel has fewer registers a thread would wait for ever, so it
// is refused instead.  Checked once per kernel.
template <auto Kern>
cudaError_t check_registers(int needed) {
  static std::atomic<int> have{-1};
  int n = have.load(std::memory_order_relaxed);
  if (n < 0) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, Kern);
    if (e != cudaSuccess) return e;
    have.store(n = at.numRegs, std::memory_order_relaxed);
  }
  return n >= needed ? cudaSuccess : cudaErrorLaunchOutOfResources;
}

}  // namespace
}  // namespace lod
