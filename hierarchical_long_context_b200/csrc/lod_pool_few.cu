// lod_pool_few.cu -- exact attention of few new tokens (at most 64 query rows per
// sequence and KV head, 32 of an 8-bit pool) over the block pool: the cache streams past once.
#include "lod_pool_list.cuh"
#include "lod_pool_tc.cuh"

namespace lod {
namespace {

template <int D, int RQ, bool Q8>
struct FewSmem {
  static constexpr int NQ = RQ < 16 ? 16 : RQ;  // the MMAs' N (a multiple of 16 with M = 128)
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kWide = D == 64 ? 2 : 1;  // d = 64 has room for twice the stages
  // stages: what 227 KB hold beside the query and weight tiles.  (8-bit, at
  // most 16 rows: two f16 tiles of each kind and two of codes, not one and
  // three: with one the conversion of a tile waits for the MMAs of the last)
  static constexpr int KS = kWide * (Q8 ? (RQ <= 16 ? 2 : 1) : RQ == 64 ? 2 : 3);
  static constexpr int VS = kWide * (Q8 ? 2 : RQ >= 32 ? 2 : 3);
  static constexpr int RS = kWide * 2;  // stages of codes (K and V of a tile)
  static constexpr int kRaw = 128 * D;  // codes of a tile
  static constexpr int kQ = NQ * D * 2, kP = NQ * 256;
  static constexpr size_t off_V = 0;  // (with d = 64 MMA 2 reads one tile past a V tile: K tiles follow)
  static constexpr size_t off_K = off_V + (size_t)VS * kTile;
  static constexpr size_t off_P = off_K + (size_t)KS * kTile;  // [2][2 key halves][NQ][128 B]
  static constexpr size_t off_Q = off_P + 2 * kP;              // [2][D / 64 halves][NQ][128 B]
  static constexpr size_t off_raw = off_Q + 2 * kQ;
  static constexpr size_t off_ex = off_raw + (Q8 ? (size_t)RS * 2 * kRaw : 0);  // uint8 [16][2][128]
  static constexpr size_t off_m = off_ex + (Q8 ? 16 * 256 : 0);       // float [2][64]
  static constexpr size_t off_red = off_m + 2 * 4 * 64;               // float [2][4][64]
  static constexpr size_t off_fin = off_red + 2 * 4 * 4 * 64;         // float2 [64]
  static constexpr size_t off_qe = off_fin + 8 * 64;                  // float [16][NQ]
  static constexpr size_t off_pos = off_qe + (Q8 ? 16 * 4 * NQ : 0);  // int2 [2][64]
  static constexpr size_t off_info = off_pos + 2 * 8 * 64;                          // uint32 [16]
  static constexpr size_t off_wb = off_info + 64;                               // int64 [kInlineSeqs + 1]
  static constexpr int kBars = 2 * KS + 2 * VS + 2 * 2 * RS + 2 + 2 + 2 + 2 + 4 + 16 + 2;
  static constexpr size_t off_bar = off_wb + 8 * (kInlineSeqs + 1);
  static constexpr size_t bytes = off_bar + 8 * kBars + 48 + 1024;  // (TMEM slot, abort flag, scales)
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // block masks, exponent bytes and query scales are kept for 16 tiles (units
  // have one at least): the copies run at
  // most RS tiles ahead of the codes' warps, and those (or, without codes,
  // the copies) KS + 2 (K) or VS (V) tiles ahead of the softmax
  static_assert(RS + (KS + 2 > VS ? KS + 2 : VS) < 16, "ring of block masks and exponents");
};

// The cache is the A operand: S^T = K Q^T (M = 128 keys, N = query rows), so
// a thread of the softmax owns a key, an 8-bit row's exponent is one factor
// of that thread, and few query rows cost few columns rather than a padded
// tile of 128 rows; O^T += V^T P^T (M = channels).  A tile's weights are
// taken against a reference maximum per query row; only when some score
// exceeds it by more than 2^8 (and on a unit's first tile) does the
// warpgroup find new maxima and rescale O^T.
// With an 8-bit pool the weight of a key carries its value row's exponent e_v
// relative to cv, the largest of the warpgroup's first tile: w = 2^(score + dv
// - m), dv = e_v - cv, with m the running maximum of score + dv.  The codes
// then enter the MMA as they are, and w fills f16's range from the top, so
// what f16 drops lies 2^-30 below the largest weighted value.  The sums take
// w 2^-dv, and so need w in fp32's range: dv is held at or above -60, and a
// row smaller than that takes the rest as a factor behind the exponential
// (rows of zeros are the common case; a first tile of nothing else has cv =
// 0).
// Roles: warp 0 copies of keys, warp 1 the MMAs of S^T, warp 2 those of O^T
// (two issuers: neither waits for the other's operands), warp 3 query tiles
// and copies of values, warps 4-7 and 8-11 the softmax of even and odd tiles,
// each with maxima, sums and an O^T of its own (a tile's chain of waits,
// loads, exponentials and stores measured 1600 to 3000 cycles, more than its
// bytes take, so two chains run side by side and are joined at the unit's
// end), with an 8-bit pool warps 12-15 and 16-19 codes to f16 (keys, values).
// Bounds: the cache's bytes, 64 KB a tile (bf16, d = 128) at 1/148 of the HBM
// rate, 1.5 us; the tensor work is below a tenth of that.  Measured at 4 x 64K
// tokens, 64 / 8 heads, one new token: bf16 168 us (6.38 TB/s, 97 % of the
// measured copy rate), d = 64 95 us (5.63 TB/s), four new tokens 195 us.
// 8-bit: 130 us (4.15 TB/s).  There the codes and f16 tiles that go in and out
// of shared memory, 192 KB a tile, take 1500 cycles of it (the load and store
// instructions' part reads 32 % of that pipe), against 1400 for the bytes from
// HBM, and the conversion and softmax chains share the rest.
template <int D, int RQ, bool Q8>
__global__ void __launch_bounds__(Q8 ? 640 : 384, 1)
    pool_few_kernel(const __grid_constant__ PoolMaps maps, const __grid_constant__ PoolAttendArgs a) {
  using S = FewSmem<D, RQ, Q8>;
  constexpr int NQ = S::NQ, KS = S::KS, VS = S::VS, RS = S::RS;
  constexpr float kTau = 8.f;
  constexpr float kUp = 6.f;  // 8-bit: weights are up to 2^14 of f16's 2^16
  constexpr int kDvMin = -60, kDvMax = 126, kNoRow = -256;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + S::off_bar);
  uint64_t* kempty = kfull + KS;
  uint64_t* vfull = kempty + KS;
  uint64_t* vempty = vfull + VS;
  uint64_t* raw_full = vempty + VS;       // [RS][2]
  uint64_t* raw_empty = raw_full + 2 * RS;
  uint64_t* s_full = raw_empty + 2 * RS;  // [2]
  uint64_t* s_free = s_full + 2;
  uint64_t* p_ready = s_free + 2;
  uint64_t* pv_done = p_ready + 2;
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_empty = q_full + 2;
  uint64_t* ex_full = q_empty + 2;  // [16] a tile's block mask and exponent bytes
  uint64_t* fin = ex_full + 16;     // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 2);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* m_s = reinterpret_cast<float*>(sm + S::off_m);
  float* red_s = reinterpret_cast<float*>(sm + S::off_red);
  int2* pos_s = reinterpret_cast<int2*>(sm + S::off_pos);
  uint32_t* info_s = reinterpret_cast<uint32_t*>(sm + S::off_info);  // blocks that are there
  float* qe_s = reinterpret_cast<float*>(sm + S::off_qe);
  float* up_s = reinterpret_cast<float*>(const_cast<int*>(abort_s) + 1);
  unsigned char* ex_s = sm + S::off_ex;
  int64_t* wb_s = reinterpret_cast<int64_t*>(sm + S::off_wb);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 32) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&kfull[i], Q8 ? 4 : 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&vfull[i], Q8 ? 4 : 1);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < 2 * RS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_ready[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&fin[i], 1);
    }
    for (int i = 0; i < 16; ++i) mbar_init(&ex_full[i], Q8 ? 33 : 1);
    *abort_s = 0;
    fence_mbar_init();
    if (!Q8) {
      tc::prefetch_tensormap(&maps.K);
      tc::prefetch_tensormap(&maps.V);
    }
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, 256);
  for (int i = tid; i < 2 * S::kP / 16; i += blockDim.x)  // rows of P past RQ stay zero
    reinterpret_cast<uint4*>(sm + S::off_P)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async();
  const int64_t* Wb = a.Wb;
  if (a.planned) pdl_wait();  // (the plan)
  if (!a.planned) {
    plan_inline<RQ, kKT>(a, wb_s);
    Wb = wb_s;
  }
  clear_refused<__nv_bfloat16, D, true>(a, Wb);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColO = 128;  // S^T in columns [0, 64) and [64, 128), O^T of even and odd tiles behind them

  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_or_abort(bar, parity, abort_s, a.status); };
  // wait for use number `i` of a ring of n barriers
  auto wait_ring = [&](uint64_t* bars, int n, int i) { return wait(&bars[i % n], (uint32_t)(i / n) & 1u); };
  const int shift = a.pool.shift;
  const int per_tile = kKT >> shift;
  const uint32_t all_ok = (per_tile == 32 ? 0xffffffffu : (1u << per_tile) - 1);

  // The copies of a unit's keys (kv = 0) or values (kv = 1); `c` counts key
  // tiles.  The values' warp also gives the softmax each tile's block mask and,
  // of an 8-bit pool, the exponent bytes of keys and values (one 16-byte copy
  // of 16 lanes; as bulk copies of a block's bytes they took as long to issue
  // as the codes), with a barrier of their own: the softmax then starts on
  // scores while the tile's values are still being converted.
  auto copies = [&](const Walk<RQ, kKT>& w, int kv, int& c) -> bool {
    Feed f(a, w.u.b, w.s.len, w.kt0, w.kt1);
    const int n = Q8 ? RS : kv ? VS : KS;
    const uint8_t* codes = static_cast<const uint8_t*>(kv ? a.pool.V : a.pool.K);
    const CUtensorMap* map = kv ? &maps.V : &maps.K;
    const int Hkv = a.pool.Hkv, h = w.u.h;
    for (int kt = w.kt0; kt < w.kt1; f.advance(), ++kt, ++c) {
      const unsigned ok = __ballot_sync(0xffffffffu, f.cur >= 0);
      const int rows = __popc(ok) << shift;
      const int row = (f.cur * Hkv + h) << shift;  // (a pool has fewer than 2^31 rows)
      const int st = c % n;
      uint64_t* full = Q8 ? &raw_full[st * 2 + kv] : (kv ? vfull : kfull) + st;
      if (c >= n && !wait(Q8 ? &raw_empty[st * 2 + kv] : (kv ? vempty : kempty) + st, (uint32_t)(c / n - 1) & 1u))
        return false;
      if (kv == 1) {
        if constexpr (Q8) {
          const int x = (lane & 7) * 16;
          const int e = __shfl_sync(0xffffffffu, f.cur, x >> shift);
          if (lane < 16) {
            const uint8_t* from = (lane < 8 ? a.pool.Ke : a.pool.Ve);
            const bool there = e >= 0;
            cp_async16_zfill(ex_s + (c & 15) * 256 + lane * 16,
                             there ? from + (((int64_t)e * Hkv + h) << shift) + (x & ((1 << shift) - 1)) : from, there);
          }
          cp_async_mbar_arrive_noinc(&ex_full[c & 15]);
        }
        if (lane == 0) {
          info_s[c & 15] = ok;
          mbar_arrive(&ex_full[c & 15]);
        }
      }
      if (lane == 0) {
        if (rows) mbar_arrive_expect(full, (uint32_t)rows * D * (Q8 ? 1 : 2));
        else mbar_arrive(full);
      }
      __syncwarp();
      if (f.cur >= 0) {
        if constexpr (Q8) {
          bulk_g2s(sm + S::off_raw + (st * 2 + kv) * S::kRaw + (lane << shift) * D, codes + (int64_t)row * D,
                   (uint32_t)D << shift, full);
        } else {
          unsigned char* d = sm + (kv ? S::off_V : S::off_K) + (size_t)st * S::kTile + (lane << shift) * 128;
          tma_load_box(d, map, 0, row, full);
          if (D == 128) tma_load_box(d + kHalfBytes, map, 64, row, full);
        }
      }
    }
    return true;
  };
  // after a wait has given up: copies still in flight land before the CTA ends
  auto drain = [&](int kv, int c) {
    if (Q8) cp_async_wait_all();
    __syncwarp();
    if (!*abort_s || lane != 0) return;
    const int n = Q8 ? RS : kv ? VS : KS;
    for (int i = c - 1; i >= 0 && i >= c - n; --i)
      (void)mbar_wait(Q8 ? &raw_full[(i % n) * 2 + kv] : (kv ? vfull : kfull) + i % n, (uint32_t)(i / n) & 1u, a.status);
  };

  if (warp < 4) regs_dec<72>();
  if (warp == 0) {
    // ============================================================== keys
    int c = 0;
    bool go = true;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) go = copies(w, 0, c);
    drain(0, c);
  } else if (warp == 1) {
    // ============================================================== S^T = K Q^T
    {
      const uint32_t lead = elect_one();
      const uint32_t idS = Q8 ? idesc_f16(128, NQ, false, false) : tc::idesc_bf16(128, NQ, false, false);
      const uint32_t qb = smem_u32(sm + S::off_Q), kb = smem_u32(sm + S::off_K);
      int c = 0, k = 0;  // key tiles, units
      bool go = true;
      Walk<RQ, kKT> w(a, Wb, blockIdx.x);
      for (; w.more() && go; w.next(), ++k) {
        if (!(go = __all_sync(0xffffffffu, wait_ring(q_full, 2, k)))) break;
        const uint64_t qd = tc::desc_kmajor_sw128(qb + (uint32_t)(k & 1) * S::kQ);
        const int T = w.kt1 - w.kt0;
        for (int j = 0; j < T; ++j, ++c) {
          if (!(go = __all_sync(0xffffffffu, (c < 2 || wait_ring(s_free, 2, c - 2)) && wait_ring(kfull, KS, c)))) break;
          tc::fence_after_sync();
          const uint64_t kd = tc::desc_kmajor_sw128(kb + (uint32_t)(c % KS) * S::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // (the address field of a descriptor counts 16 bytes)
            mma_ss(lead, tmem + (c & 1) * 64, kd + (((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4),
                         qd + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idS, kk > 0);
          mma_commit_if(lead, &s_full[c & 1]);
          mma_commit_if(lead, &kempty[c % KS]);
          if (j == T - 1) mma_commit_if(lead, &q_empty[k & 1]);
        }
      }
      if (lane == 0) w.record(blockIdx.x);
      if (c > 0) {
        mma_commit_if(lead, &fin[0]);
        (void)mbar_wait(&fin[0], 0, a.status);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ============================================================== O^T += V^T P^T
    {
      const uint32_t lead = elect_one();
      const uint32_t idO = Q8 ? idesc_f16(128, NQ, true, false) : tc::idesc_bf16(128, NQ, true, false);
      const uint32_t pb = smem_u32(sm + S::off_P), vb = smem_u32(sm + S::off_V);
      int c = 0;
      bool go = true;
      for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) {
        const int T = w.kt1 - w.kt0;
        for (int j = 0; j < T; ++j, ++c) {
          if (!(go = __all_sync(0xffffffffu, wait_ring(vfull, VS, c) && wait_ring(p_ready, 2, c)))) break;
          tc::fence_after_sync();
          const uint64_t vd = tc::desc_mnmajor_sw128(vb + (uint32_t)(c % VS) * S::kTile, kHalfBytes);
          const uint64_t pd = tc::desc_kmajor_sw128(pb + (uint32_t)(c & 1) * S::kP);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(lead, tmem + kColO + (c & 1) * 64, vd + kk * (2048 >> 4),
                         pd + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idO, j > 1 || kk > 0);
          mma_commit_if(lead, &pv_done[c & 1]);
          mma_commit_if(lead, &vempty[c % VS]);
        }
      }
      if (c > 0) {
        mma_commit_if(lead, &fin[1]);
        (void)mbar_wait(&fin[1], 0, a.status);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ============================================================== query tiles, values
    int k = 0, c = 0;
    bool go = true;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next(), ++k) {
      if (k >= 2 && !(go = __all_sync(0xffffffffu, wait_ring(q_empty, 2, k - 2)))) break;
      unsigned char* qs = sm + S::off_Q + (size_t)(k & 1) * S::kQ;
      auto row_of = [&](int r) {
        const int g = (int)w.u.i * RQ + r;
        return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (w.s.r0 + g / a.G) * a.qt +
                                              (int64_t)(w.u.h * a.G + g % a.G) * a.qh);
      };
      if constexpr (Q8) {  // a row is a group of D / 8 lanes, 16 bytes each
        constexpr int LPR = D / 8;
        for (int r = lane / LPR; r < NQ; r += 32 / LPR) {
          const int ch = lane % LPR;
          uint4 v = r < w.nrow ? row_of(r)[ch] : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = query_exponent(top);
          const float f = exp2i(-e);
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = pack_f16x2(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xffff0000u) * f);
          *reinterpret_cast<uint4*>(qs + (ch >> 3) * NQ * 128 + sw_off(r, ch)) = make_uint4(y[0], y[1], y[2], y[3]);
          if (ch == 0) qe_s[(k & 15) * NQ + r] = exp2i(e);
        }
      } else {
        for (int x = lane; x < NQ * (D / 8); x += 32) {
          const int r = x / (D / 8), ch = x % (D / 8);
          *reinterpret_cast<uint4*>(qs + (ch >> 3) * NQ * 128 + sw_off(r, ch)) =
              r < w.nrow ? row_of(r)[ch] : make_uint4(0, 0, 0, 0);
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[k & 1]);
      go = copies(w, 1, c);
    }
    drain(1, c);
  } else if (warp < 12) {
    // ============================================================== softmax
    regs_inc<Q8 ? 136 : 216>();
    const int half = (warp - 4) >> 2;  // this warpgroup takes the tiles of this parity
    const int r = tid & 127;           // key of the tile; channel of O^T
    const int q4 = warp & 3;
    const uint32_t tl = (uint32_t)(32 * q4) << 16;
    const uint32_t ts = tmem + tl + half * 64, to = tmem + tl + kColO + half * 64;
    const int bar_or = 1 + 2 * half, bar_wg = 2 + 2 * half;  // named barriers of the warpgroup
    constexpr int kBarBoth = 5;                              // and of the two
    constexpr int CH = RQ < 16 ? 8 : 16;                     // columns of a TMEM load
    auto load_cols = [&](uint32_t at, float (&v)[CH]) {
      if constexpr (CH == 8) tc::tmem_ld8(at, v);
      else tc::tmem_ld16(at, v);
    };
    float* mine_m = m_s + half * 64;
    float* red = red_s + half * 256;
    int2* pos = pos_s + half * 64;
    int c0 = 0, k = 0;  // the unit's first tile, units
    bool go = true;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more(); w.next(), ++k) {
      const int T = w.kt1 - w.kt0;
      const float* qe = qe_s + (k & 15) * NQ;
      int cv = 0;  // (8-bit) the value exponent that O^T is in units of
      const int p0 = (int)(w.s.len - w.s.n), g0 = (int)w.u.i * RQ;
      const int pos_lo = p0 + g0 / a.G, pos_hi = p0 + (g0 + w.nrow - 1) / a.G;
      auto first_of = [&](int p) { return a.window > 0 && p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0; };
      const int first_lo = first_of(pos_lo), first_hi = first_of(pos_hi);
      if (r < RQ) {
        const int p = p0 + (g0 + (r < w.nrow ? r : w.nrow - 1)) / a.G;
        pos[r] = make_int2(first_of(p), p);  // the row's keys
        mine_m[r] = -INFINITY;
      }
      bar_named_sync(bar_wg, 128);
      float l[RQ];
#pragma unroll
      for (int n = 0; n < RQ; ++n) l[n] = 0.f;
      const int j0 = (c0 ^ half) & 1;  // this warpgroup's first tile of the unit
      for (int j = j0; j < T; j += 2) {
        const int c = c0 + j, k0 = (w.kt0 + j) * kKT, t = k0 + r;
        // (8-bit: the values too.  Conversion and softmax then take turns at the
        // shared memory, which bounds both; side by side they measured 6 % more.)
        go = __all_sync(0xffffffffu, (c < 2 || wait_ring(pv_done, 2, c - 2)) && wait_ring(ex_full, 16, c) &&
                                         (!Q8 || wait_ring(vfull, VS, c)) && wait_ring(s_full, 2, c));
        // (a failed wait is carried to the barrier below, where the four warps leave together)
        const uint32_t ok = info_s[c & 15];
        const bool masked = k0 + 127 > pos_lo || k0 < first_hi || ok != all_ok;
        bool live = true;
        int ve = 0;  // (8-bit) the value row's exponent; kNoRow: any will do, its codes are NaN
        float ks = a.scale_log2;
        if constexpr (Q8) {
          const int e0 = ex_s[(c & 15) * 256 + r], e1 = ex_s[(c & 15) * 256 + 128 + r];
          ks *= exp2i(e0 == 255 ? 0 : max(e0, 7) - 127);
          ve = e1 == 255 ? kNoRow : max(e1, 7) - 127;
        }
        float dv = 0.f, pe = 1.f, pv = 1.f;  // (pe: a weight to the sums' unit; pv: what dv lacks of the row's exponent)
        if constexpr (Q8) {
          if (j == j0) {
            // cv, by each warp from the tile's bytes: four a lane, those of
            // NaN rows, behind the length and before every window left out
            const uint32_t e4 = reinterpret_cast<const uint32_t*>(ex_s + (c & 15) * 256 + 128)[lane];
            const int there = (int)w.s.len - k0 - 4 * lane, before = first_lo - k0 - 4 * lane;
            uint32_t b4 = e4 & ~__vcmpeq4(e4, 0xffffffffu);
            b4 &= there <= 0 ? 0u : there >= 4 ? 0xffffffffu : (1u << (8 * there)) - 1;
            b4 &= before <= 0 ? 0xffffffffu : before >= 4 ? 0u : 0xffffffffu << (8 * before);
            b4 = __vmaxu4(b4, b4 >> 16);
            const int top = (int)__reduce_max_sync(0xffffffffu, __vmaxu4(b4, b4 >> 8) & 0xff);
            cv = top <= 7 ? 0 : top - 127;
          }
          const int dt = ve - cv, d = min(max(dt, kDvMin), kDvMax);
          dv = (float)d;
          pe = exp2i(-d);
          pv = ve == kNoRow ? 1.f : exp2i(min(max(dt - d, -126), 0));
        }
        if (masked) {
          live = t < w.s.len && ((ok >> (r >> shift)) & 1u);
          // (a barrier's parity tells a phase only from the one before it: with
          // the sums of tile c - 2 complete, V_{c - VS} has landed)
          static_assert(VS >= 2, "wait for the values");
          go = go && __all_sync(0xffffffffu, wait_ring(vfull, VS, c));
          if (go && (!live || t < first_lo)) {
            // no row's key: the weights' zeros must not meet what the pool
            // holds there, or what shared memory held before
            unsigned char* v = sm + S::off_V + (size_t)(c % VS) * S::kTile;
#pragma unroll
            for (int q = 0; q < D / 8; ++q)
              *reinterpret_cast<uint4*>(v + (q >> 3) * kHalfBytes + sw_off(r, q)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        tc::fence_after_sync();
        float y[RQ];
#pragma unroll
        for (int n0 = 0; n0 < RQ; n0 += CH) {
          float v[CH];
          load_cols(ts + n0, v);
#pragma unroll
          for (int n = 0; n < CH; ++n) y[n0 + n] = v[n] * (Q8 ? ks * qe[n0 + n] : ks);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[half]);
        if (masked) {
#pragma unroll
          for (int n = 0; n < RQ; ++n) {
            const int2 fl = pos[n];
            y[n] = live && t >= fl.x && t <= fl.y ? y[n] : -INFINITY;
          }
        }
        bool grow = j == j0 || !go;
        const float tau = kTau - dv;
#pragma unroll
        for (int n = 0; n < RQ; n += 4) {
          const float4 mr = *reinterpret_cast<const float4*>(mine_m + n);
          grow |= y[n] > mr.x + tau || y[n + 1] > mr.y + tau || y[n + 2] > mr.z + tau || y[n + 3] > mr.w + tau;
        }
        if (bar_red_or(bar_or, 128, grow)) {
          go = !bar_red_or(bar_or, 128, !go);
          if (!go) break;
          // new maxima: over the warp's keys, then over the four warps (the
          // sums of tile c - 2 are complete: waited for above)
#pragma unroll
          for (int n = 0; n < RQ; ++n) {
            const float x = warp_max(y[n] + dv);
            if (lane == n % 32) red[q4 * 64 + n] = x;
          }
          bar_named_sync(bar_wg, 128);
#pragma unroll
          for (int n0 = 0; n0 < RQ; n0 += 8) {
            float f[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const int q = n0 + n;
              const float x = fmaxf(fmaxf(red[q], red[64 + q]), fmaxf(red[128 + q], red[192 + q]));
              const float m = mine_m[q];
              f[n] = x > m ? (m == -INFINITY ? 0.f : ex2_approx(m - x)) : 1.f;
              l[q] *= f[n];
            }
            if (j > j0) {
              float o[8];
              tc::tmem_ld8(to + n0, o);
#pragma unroll
              for (int n = 0; n < 8; ++n) o[n] *= f[n];
              tc::tmem_st8(to + n0, o);
            }
          }
          bar_named_sync(bar_wg, 128);  // every thread has read the old maxima
          if (r < RQ)
            mine_m[r] = fmaxf(fmaxf(fmaxf(red[r], red[64 + r]), fmaxf(red[128 + r], red[192 + r])), mine_m[r]);
          bar_named_sync(bar_wg, 128);
        }
        // weights
        unsigned char* P = sm + S::off_P + (size_t)half * S::kP + (r >> 6) * NQ * 128 + (r & 7) * 2;
        const int ch = (r & 63) >> 3;
#pragma unroll
        for (int n = 0; n < RQ; n += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(mine_m + n);
          const float mr[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p = ex2_approx(y[n + q] - (mr[q] == -INFINITY ? 0.f : mr[q]) + (Q8 ? dv + kUp : 0.f));
            l[n + q] = Q8 ? fmaf(p, pe, l[n + q]) : l[n + q] + p;
            *reinterpret_cast<uint16_t*>(P + (n + q) * 128 + ((ch ^ ((n + q) & 7)) << 4)) =
                Q8 ? (uint16_t)pack_f16x2(p * pv, 0.f) : (uint16_t)pack_bf16x2(p, 0.f);
          }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[half]);
      }
      // ---- the unit's result, or this CTA's piece of it: warpgroup 1 hands
      // its maxima and sums over, warpgroup 0 joins both
      const int mine = (T - j0 + 1) >> 1;  // this warpgroup's tiles
      if (go && mine > 0) go = __all_sync(0xffffffffu, wait_ring(pv_done, 2, c0 + j0 + 2 * (mine - 1)));
      tc::fence_after_sync();
#pragma unroll
      for (int n = 0; n < RQ; ++n) {
        const float x = warp_sum(l[n]);
        if (lane == n % 32) red[q4 * 64 + n] = x;
      }
      bar_named_sync(bar_wg, 128);
      // 8-bit: the sums are in units of 2^(m - kUp), O^T of 2^(m - kUp + cv)
      const float dm = Q8 ? kUp : 0.f;
      float2* fin_s = reinterpret_cast<float2*>(sm + S::off_fin);
      const float up = Q8 ? exp2i(cv) : 1.f;
      if (half == 1) {
        if (r < RQ)
          fin_s[r] = make_float2(mine_m[r] - dm, (red[r] + red[64 + r]) + (red[128 + r] + red[192 + r]));
        if (r == 0) up_s[0] = mine > 0 ? up : 0.f;
      }
      go = !bar_red_or(kBarBoth, 256, !go);
      if (!go) break;
      if (half == 0) {
        const bool whole = w.whole();
        const int64_t at = (int64_t)w.slot(blockIdx.x) * RQ;
        const float up1 = up_s[0];
#pragma unroll 1
        for (int n0 = 0; n0 < RQ; n0 += 8) {
          float o[8], o1[8];
          tc::tmem_ld8(to + n0, o);
          tc::tmem_ld8(to + 64 + n0, o1);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int row = n0 + n;
            if (row < w.nrow) {
              const float2 f1 = fin_s[row];
              const float m0 = mine_m[row] - dm, l0 = (red[row] + red[64 + row]) + (red[128 + row] + red[192 + row]);
              const float m = fmaxf(m0, f1.x), ref = m == -INFINITY ? 0.f : m;
              const float a0 = ex2_approx(m0 - ref), a1 = ex2_approx(f1.x - ref);
              const float sum = fmaf(l0, a0, f1.y * a1);
              // (a warpgroup without a tile has nothing in its O^T)
              const float x = (mine > 0 ? o[n] * (up * a0) : 0.f) + (up1 != 0.f ? o1[n] * (up1 * a1) : 0.f);
              const int g = g0 + row, tok = g / a.G, head = w.u.h * a.G + g % a.G;
              if (whole) {
                const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
                if (r < D)
                  (static_cast<__nv_bfloat16*>(a.out) + (w.s.r0 + tok) * a.ot + (int64_t)head * a.oh)[r] =
                      __float2bfloat16_rn(x * inv);
                if (r == 0 && a.lse)
                  a.lse[(w.s.r0 + tok) * a.Hq + head] = (m + log2f(sum)) * 0.6931471805599453f;
              } else {
                if (r < D) a.part[(at + row) * D + r] = x;
                if (r == 0) a.ml[at + row] = make_float2(m, sum);
              }
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      bar_named_sync(kBarBoth, 256);  // both O^T, fin_s and up_s have been read
      c0 += T;
    }
  } else if constexpr (Q8) {
    // ============================================================== codes to f16 tiles
    regs_dec<64>();
    int c = 0;
    bool go = true;
    const int kv = (warp - 12) >> 2, n = kv ? VS : KS;
    uint64_t* full = kv ? vfull : kfull;
    uint64_t* empty = kv ? vempty : kempty;
    unsigned char* ring = sm + (kv ? S::off_V : S::off_K);
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) {
      for (int j = w.kt0; j < w.kt1; ++j, ++c) {
        const int raw = (c % RS) * 2 + kv;
        go = __all_sync(0xffffffffu, wait(&raw_full[raw], (uint32_t)(c / RS) & 1u) &&
                                         (c < n || wait(&empty[c % n], (uint32_t)(c / n - 1) & 1u)));
        if (!go) break;
        // (the rows' powers of two are left to the softmax)
        convert_tile<D, false>(sm + S::off_raw + raw * S::kRaw, nullptr, ring + (size_t)(c % n) * S::kTile, tid & 127);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[raw]);
          mbar_arrive(&full[c % n]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 256);
}

template <int D, int RQ, bool Q8>
cudaError_t launch_few(const PoolAttendArgs& a, const PoolMaps* maps, cudaStream_t st) {
  using S = FewSmem<D, RQ, Q8>;
  cudaError_t e = set_smem_once<pool_few_kernel<D, RQ, Q8>>(S::bytes);
  // 128 (72 + 216 + 216) = 384 * 168 and 128 (72 + 136 + 136 + 64 + 64) < 640 * 96
  if (e == cudaSuccess) e = check_registers<pool_few_kernel<D, RQ, Q8>>(Q8 ? 96 : 168);
  if (e == cudaSuccess && a.planned) e = launch_plan<RQ, kKT>(a, st);
  if (e != cudaSuccess) return e;
  PoolMaps none = {};
  const dim3 grid(a.ctas), block(Q8 ? 640 : 384);
  if (a.planned) {
    e = launch_pdl(pool_few_kernel<D, RQ, Q8>, grid, block, S::bytes, st, maps ? *maps : none, a);
  } else {
    pool_few_kernel<D, RQ, Q8><<<grid, block, S::bytes, st>>>(maps ? *maps : none, a);
    e = cudaGetLastError();
  }
  return e != cudaSuccess ? e : launch_merge<__nv_bfloat16, D, RQ, kKT>(a, st);
}

template <int D, bool Q8>
cudaError_t launch_few_d(const PoolAttendArgs& a, const PoolMaps* maps, int TM, cudaStream_t st) {
  switch (TM) {
    case 8: return launch_few<D, 8, Q8>(a, maps, st);
    case 16: return launch_few<D, 16, Q8>(a, maps, st);
    case 32: return launch_few<D, 32, Q8>(a, maps, st);
    default:
      if constexpr (!Q8) return launch_few<D, 64, Q8>(a, maps, st);
      return cudaErrorInvalidValue;  // (pool_shape gives more than 32 rows of an 8-bit pool to the other kernel)
  }
}

}  // namespace

cudaError_t launch_pool_few(const PoolAttendArgs& a, const PoolMaps* maps, int TM, int bits, int d, cudaStream_t stream) {
  if (d == 64) return bits == 8 ? launch_few_d<64, true>(a, maps, TM, stream) : launch_few_d<64, false>(a, maps, TM, stream);
  return bits == 8 ? launch_few_d<128, true>(a, maps, TM, stream) : launch_few_d<128, false>(a, maps, TM, stream);
}

}  // namespace lod
