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

__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return done;
}
// Bounded wait for phase `parity` of `bar`; false once a wait of the CTA has
// given up (abort_s), which a wait of about a second does.  The flag is looked
// at only when the phase is not complete yet: a role waits several times a
// key tile, and mostly for what has long happened.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_s, uint32_t* status) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!*abort_s) {
    if (mbar_try(bar, parity)) return true;
    if (clock64() - t0 > (2ll << 30)) {
      set_status(status, LOD_ST_TIMEOUT);
      *abort_s = 1;
    }
  }
  return false;
}

// ---------------------------------------------------------------- block entries

// The copying warp's view of a piece's key tiles: the blocks of the present
// tile (lane i: the tile's block i, -1: none or bad) and, of an 8-bit pool,
// its exponent bytes (lanes 0-7 of the keys, 8-15 of the values, 16 tokens
// each), read one and two tiles ahead so that no copy waits for them.
template <bool Q8>
struct Feed {
  const PoolAttendArgs& a;
  const int32_t* table;
  int nblk, kt1, h, cur, nxt;
  uint4 ex;

  __device__ __forceinline__ int entry(int kt) const {
    const int per_tile = kKT >> a.pool.shift, lane = threadIdx.x & 31;
    const int i = kt * per_tile + lane;
    if (lane >= per_tile || i >= nblk || kt >= kt1) return -1;
    const int e = table[i];
    if (e >= 0 && e < a.pool.blocks) return e;
    set_status(a.status, LOD_ST_BAD_PAGE);
    return -1;
  }
  __device__ __forceinline__ uint4 exponents() const {
    const int lane = threadIdx.x & 31, x = (lane & 7) * 16;
    const int b = __shfl_sync(0xffffffffu, cur, x >> a.pool.shift);
    if (lane >= 16 || b < 0) return make_uint4(0, 0, 0, 0);
    const uint8_t* e = (lane < 8 ? a.pool.Ke : a.pool.Ve) + (((int64_t)b * a.pool.Hkv + h) << a.pool.shift);
    return *reinterpret_cast<const uint4*>(e + (x & ((1 << a.pool.shift) - 1)));
  }
  __device__ __forceinline__ Feed(const PoolAttendArgs& args, int b, int head, int64_t len, int kt0, int end)
      : a(args), table(args.batch.table + (int64_t)b * args.batch.max_blocks),
        nblk((int)((len + (1 << args.pool.shift) - 1) >> args.pool.shift)), kt1(end), h(head) {
    cur = entry(kt0);
    nxt = entry(kt0 + 1);
    if (Q8) ex = exponents();
  }
  __device__ __forceinline__ void advance(int kt) {  // from tile kt to kt + 1
    cur = nxt;
    nxt = entry(kt + 2);
    if (Q8) ex = exponents();
  }
};

// ---------------------------------------------------------------- e4m3 -> bf16

// Four e4m3 codes as four bf16 (two words), times f.  Shifted into a bf16's
// exponent and mantissa, a code's low seven bits read as the code's value
// times 2^-120 (bias 127 against 7; a subnormal code becomes a subnormal
// bf16), so a product by 2^120 gives the value, exactly.
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t f, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  lo = hmul2_bf16(((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), f);
  hi = hmul2_bf16(((b >> 4) & 0x07f007f0u) | (b & 0x80008000u), f);
}
// 2^120 2^(E - 127) in two factors (it can leave bf16's range), each in both
// halves of a word; E = 255: NaN.  The pool never holds E below 7; smaller
// ones read as 7.
__device__ __forceinline__ void e4m3_factors(int E, uint32_t& f1, uint32_t& f2) {
  const int e = (E < 7 ? 7 : E) - 127, e1 = e < 7 ? e : 7;
  const uint32_t a = (uint32_t)(e1 + 120 + 127) << 7, b = E == 255 ? 0x7fc0u : (uint32_t)(e - e1 + 127) << 7;
  f1 = a | (a << 16);
  f2 = b | (b << 16);
}

// A tile of 128 rows of codes (src, rows of D bytes; ex: their exponent
// bytes) as a bf16 tile in the 128-byte-swizzled layout, by 128 threads
// (t < 128).  SCALED: times the rows' powers of two; else the codes' values.
// A thread converts 16 codes of every (128 / (D / 16))-th row, so its place in
// the swizzle is the same for all of them.  With D = 128 a row's two halves
// lie on the same banks: the second half's threads store their two chunks in
// the other order.
template <int D, bool SCALED>
__device__ __forceinline__ void convert_tile(const unsigned char* src, const unsigned char* ex, unsigned char* dst, int t) {
  constexpr int CPR = D / 16, RPI = 128 / CPR, IT = 128 / RPI;
  const int row0 = t / CPR, ch = t % CPR;
  const bool swap = D == 128 && (ch & 4);
  unsigned char* d = dst + (ch >> 2) * kHalfBytes;
  const uint32_t o0 = sw_off(row0, 2 * ch + (swap ? 1 : 0)), o1 = sw_off(row0, 2 * ch + (swap ? 0 : 1));
  constexpr int BATCH = 4;
#pragma unroll
  for (int i0 = 0; i0 < IT; i0 += BATCH) {
    uint4 v[BATCH];
    int E[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      v[i] = *reinterpret_cast<const uint4*>(src + (t + 128 * (i0 + i)) * 16);
      if (SCALED) E[i] = ex[row0 + RPI * (i0 + i)];
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t w[4] = {swap ? v[i].z : v[i].x, swap ? v[i].w : v[i].y, swap ? v[i].x : v[i].z,
                             swap ? v[i].y : v[i].w};
      uint32_t x[8];
      uint32_t f1 = 0x7b807b80u, f2 = 0;
      if (SCALED) e4m3_factors(E[i], f1, f2);
#pragma unroll
      for (int q = 0; q < 4; ++q) e4m3x4_bf16(w[q], f1, x[2 * q], x[2 * q + 1]);
      if (SCALED) {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = hmul2_bf16(x[q], f2);
      }
      unsigned char* r = d + (i0 + i) * RPI * 128;
      *reinterpret_cast<uint4*>(r + o0) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(r + o1) = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
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
