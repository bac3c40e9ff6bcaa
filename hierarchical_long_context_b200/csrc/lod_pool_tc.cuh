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
// The largest of three; NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^x of a pair on the FMA pipe, for x <= 128 (0 below -127; not for NaN): x =
// n + f with n the nearest integer (the sum with 1.5 * 2^23 leaves it in the
// low bits), a polynomial of degree 5 for 2^f on [-1/2, 1/2], n added to its
// exponent.  The coefficients minimise the largest relative error with
// p(0) = 1 (a linear programme over a grid): 8.1e-8, 1.6e-7 with the fp32
// roundings (degree 4: 2.9e-6, more than the bound on a weight allows).
__device__ __forceinline__ float2 exp2_fma2(float2 x) {
  constexpr float kMagic = 12582912.f;
  x.x = fmaxf(x.x, -127.f);
  x.y = fmaxf(x.y, -127.f);
  const float2 t = fadd2(x, make_float2(kMagic, kMagic));
  const float2 n = fadd2(t, make_float2(-kMagic, -kMagic));
  const float2 f = ffma2(n, make_float2(-1.f, -1.f), x);
  constexpr float c5 = 0.0013274633092805743f, c4 = 0.009671961888670921f, c3 = 0.055506784468889236f,
                  c2 = 0.24022234976291656f, c1 = 0.6931470632553101f;
  float2 p = ffma2(make_float2(c5, c5), f, make_float2(c4, c4));
  p = ffma2(p, f, make_float2(c3, c3));
  p = ffma2(p, f, make_float2(c2, c2));
  p = ffma2(p, f, make_float2(c1, c1));
  p = ffma2(p, f, make_float2(1.f, 1.f));
  p.x = __uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23));
  p.y = __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23));
  return p;
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
__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two floats rounded (RNE) to f16 and packed, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Instruction descriptor, kind::f16 with f16 inputs and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return tc::idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));  // formats 0: f16
}
// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return done;
}
// The same, the thread set aside for up to about 10 us: a role that is ahead
// of the others leaves them the issue slots.
__device__ __forceinline__ bool mbar_try_long(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
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
    if (mbar_try_long(bar, parity)) return true;
    if (clock64() - t0 > (2ll << 30)) {
      set_status(status, LOD_ST_TIMEOUT);
      *abort_s = 1;
    }
  }
  return false;
}

// MMAs and commits issued by one lane of a warp that runs its loop as a whole:
// with the lane chosen by a predicate inside the instruction's own block, the
// loop's values stay uniform over the warp and the descriptors sit in uniform
// registers.  Under an `if (lane == 0)` around the loop every operand was moved
// there first, and 8 MMAs took about 700 cycles to issue.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}\n" ::"r"(lead),
      "r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}\n" ::"r"(lead),
      "r"(d), "r"(at), "l"(bd), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}\n" ::"r"(lead),
      "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- block entries

// A copying warp's view of a piece's key tiles: the blocks of the present
// tile (lane i: the tile's block i, -1: none or bad).  A tile's copies take
// less time to issue than a table entry takes to arrive, so entries are read
// kAhead tiles ahead.
constexpr int kAhead = 4;
struct Feed {
  const PoolAttendArgs& a;
  const int32_t* next;      // this lane's entry of the tile behind the queue
  int left, per_tile, cur;  // left: entries of the sequence from `next` on
  int tiles;                // tiles of the piece behind the queue
  int ent[kAhead + 1];

  __device__ __forceinline__ int entry() {
    const int lane = threadIdx.x & 31;
    int e = INT32_MIN;
    if (lane < per_tile && lane < left && tiles > 0) e = *next;
    next += per_tile;
    left -= per_tile;
    --tiles;
    return e;
  }
  __device__ __forceinline__ void present() {
    cur = ent[0] >= 0 && ent[0] < a.pool.blocks ? ent[0] : -1;
    if (ent[0] != INT32_MIN && cur < 0) set_status(a.status, LOD_ST_BAD_PAGE);
  }
  __device__ __forceinline__ Feed(const PoolAttendArgs& args, int b, int64_t len, int kt0, int kt1)
      : a(args), per_tile(kKT >> args.pool.shift), tiles(kt1 - kt0) {
    const int nblk = (int)((len + (1 << args.pool.shift) - 1) >> args.pool.shift);
    next = args.batch.table + (int64_t)b * args.batch.max_blocks + (int64_t)kt0 * per_tile + (threadIdx.x & 31);
    left = nblk - kt0 * per_tile;
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) ent[i] = entry();
    present();
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ent[i] = ent[i + 1];
    ent[kAhead] = entry();
    present();
  }
};

// ---------------------------------------------------------------- e4m3 -> f16

// The MMAs of an 8-bit pool take f16 operands: every e4m3 value is an f16
// value, the hardware converts a pair in one instruction (into bf16 it takes
// five on the integer pipe, which measured 3.5 times as long), and f16 weights
// carry three bits more than bf16 ones.  What f16 lacks is range, so powers
// of two are taken out of every operand and put back in fp32: the queries'
// rows are scaled to a largest value in [2^14, 2^15) (what that loses lies
// 2^-39 below the row's largest), and the rows' exponents are handled as the
// kernels say.

// Factor 2^(E - C) of a row of exponent byte E in a tile whose largest is C,
// as f16 bits (a row 2^24 below the tile's largest is dropped: that is below
// the rounding of the fp32 sums it would enter).
__device__ __forceinline__ uint32_t row_factor(int E, int C) {
  const int d = E - C;
  return E == 255 || d >= 0 ? 0x3c00u : d >= -14 ? (uint32_t)(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
}

// Exponent e that brings a query row with the largest bf16 magnitude bits
// `top` to [2^14, 2^15) when multiplied by 2^-e; 0 for a row of zeros, of an
// infinity or NaN.
__device__ __forceinline__ int query_exponent(uint32_t top) {
  if (top == 0 || top >= 0x7f80u) return 0;
  const int e = (int)(top >> 7) - 127 - 14;
  return e < -126 ? -126 : e;
}
// A query row of D bf16 channels (D / 8 words) as f16 times 2^-e; returns e.
template <int D>
__device__ __forceinline__ int query_f16(uint4 (&x)[D / 8]) {
  uint32_t* w = &x[0].x;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < D / 2; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  const int e = query_exponent(top);
  const float f = exp2i(-e);
#pragma unroll
  for (int i = 0; i < D / 2; ++i)
    w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
  return e;
}

// A tile of 128 rows of codes (src, rows of D bytes) as an f16 tile in the
// 128-byte-swizzled layout, by 128 threads (t < 128); with SCALED times the
// rows' factors (fac, f16 bits).  A thread converts 16 codes of every
// (128 / (D / 16))-th row, so its place in the swizzle is the same for all of
// them.  With D = 128 a row's two halves lie on the same banks: the second
// half's threads store their two chunks in the other order.
template <int D, bool SCALED>
__device__ __forceinline__ void convert_tile(const unsigned char* src, const uint16_t* fac, unsigned char* dst, int t) {
  constexpr int CPR = D / 16, RPI = 128 / CPR, IT = 128 / RPI;
  const int row0 = t / CPR, ch = t % CPR;
  const bool swap = D == 128 && (ch & 4);
  unsigned char* d = dst + (ch >> 2) * kHalfBytes;
  const uint32_t o0 = sw_off(row0, 2 * ch + (swap ? 1 : 0)), o1 = sw_off(row0, 2 * ch + (swap ? 0 : 1));
  constexpr int BATCH = 4;
#pragma unroll
  for (int i0 = 0; i0 < IT; i0 += BATCH) {
    uint4 v[BATCH];
    uint32_t f[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      v[i] = *reinterpret_cast<const uint4*>(src + (t + 128 * (i0 + i)) * 16);
      if (SCALED) f[i] = fac[row0 + RPI * (i0 + i)] * 0x10001u;
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t w[4] = {swap ? v[i].z : v[i].x, swap ? v[i].w : v[i].y, swap ? v[i].x : v[i].z,
                             swap ? v[i].y : v[i].w};
      uint32_t x[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
            : "=r"(x[2 * q]), "=r"(x[2 * q + 1])
            : "r"(w[q]));
        if (SCALED) {
          x[2 * q] = hmul2_f16(x[2 * q], f[i]);
          x[2 * q + 1] = hmul2_f16(x[2 * q + 1], f[i]);
        }
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
