// lod_pool_few.cu -- exact attention of few new tokens (at most 64 query rows per
// sequence and KV head) over the block pool: the cache streams past once.
#include "lod_pool_list.cuh"
#include "lod_pool_tc.cuh"

namespace lod {
namespace {

template <int D, int RQ, bool Q8>
struct FewSmem {
  static constexpr int NQ = RQ < 16 ? 16 : RQ;  // the MMAs' N (a multiple of 16 with M = 128)
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kWide = D == 64 ? 2 : 1;  // d = 64 has room for twice the stages
  // stages: what 227 KB hold beside the query and weight tiles
  static constexpr int KS = kWide * (Q8 ? 1 : RQ == 64 ? 2 : 3);
  static constexpr int VS = kWide * (Q8 ? (RQ == 64 ? 1 : 2) : RQ >= 32 ? 2 : 3);
  static constexpr int RS = kWide * (RQ >= 32 ? 2 : 3);  // stages of codes (K and V of a tile)
  static constexpr int kRaw = 128 * D;
  static constexpr int kQ = NQ * D * 2, kP = NQ * 256;
  static constexpr size_t off_V = 0;  // (with d = 64 MMA 2 reads one tile past a V tile: K tiles follow)
  static constexpr size_t off_K = off_V + (size_t)VS * kTile;
  static constexpr size_t off_P = off_K + (size_t)KS * kTile;  // [2][2 key halves][NQ][128 B]
  static constexpr size_t off_Q = off_P + 2 * kP;              // [2][D / 64 halves][NQ][128 B]
  static constexpr size_t off_raw = off_Q + 2 * kQ;
  static constexpr size_t off_ex = off_raw + (Q8 ? (size_t)RS * 2 * kRaw : 0);  // uint8 [16][2][128]
  static constexpr size_t off_m = off_ex + (Q8 ? 16 * 256 : 0);                 // float [NQ]
  static constexpr size_t off_red = off_m + 4 * 64;                             // float [4][64]
  static constexpr size_t off_qe = off_red + 4 * 4 * 64;                        // float [16][NQ]
  static constexpr size_t off_pos = off_qe + (Q8 ? 16 * 4 * NQ : 0);                       // int2 [64]
  static constexpr size_t off_info = off_pos + 8 * 64;                          // uint2 [16]
  static constexpr size_t off_wb = off_info + 128;                               // int64 [kInlineSeqs + 1]
  static constexpr int kBars = 2 * KS + 2 * VS + 2 * 2 * RS + 2 + 2 + 2 + 2 + 4 + 2;
  static constexpr size_t off_bar = off_wb + 8 * (kInlineSeqs + 1);
  static constexpr size_t bytes = off_bar + 8 * kBars + 16 + 1024;
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
// With an 8-bit pool the weight of a key carries its value row's exponent,
// w = 2^(score + e_v - m) with m the running maximum of score + e_v: the
// codes then enter the MMA as they are, and w fills f16's range from the top,
// so what f16 drops lies 2^-30 below the largest weighted value.
// Roles: warp 0 copies of keys, warp 1 the MMAs of S^T, warp 2 those of O^T
// (two issuers: neither waits for the other's operands), warp 3 query tiles
// and copies of values, warps 4-7 softmax, with an 8-bit pool warps 8-11 and 12-15 codes to bf16
// (keys, values).
// Bound by the cache's bytes: 64 KB a tile (bf16, d = 128) at 1/148 of the
// HBM rate is 1.5 us, the tensor work of a tile well below a tenth of that.
template <int D, int RQ, bool Q8>
__global__ void __launch_bounds__(Q8 ? 512 : 256, 1)
    pool_few_kernel(const __grid_constant__ PoolMaps maps, const __grid_constant__ PoolAttendArgs a) {
  using S = FewSmem<D, RQ, Q8>;
  constexpr int NQ = S::NQ, KS = S::KS, VS = S::VS, RS = S::RS;
  constexpr float kTau = 8.f;
  constexpr float kUp = 6.f;  // 8-bit: weights are up to 2^14 of f16's 2^16
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
  uint64_t* fin = q_empty + 2;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 2);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* m_s = reinterpret_cast<float*>(sm + S::off_m);
  float* red_s = reinterpret_cast<float*>(sm + S::off_red);
  int2* pos_s = reinterpret_cast<int2*>(sm + S::off_pos);
  uint2* info_s = reinterpret_cast<uint2*>(sm + S::off_info);  // blocks that are there, largest value exponent
  float* qe_s = reinterpret_cast<float*>(sm + S::off_qe);
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
  if (!a.planned) {
    plan_inline<RQ, kKT>(a, wb_s);
    Wb = wb_s;
  }
  clear_refused<__nv_bfloat16, D>(a);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColO = 128;  // S^T in columns [0, 64) and [64, 128)

  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_or_abort(bar, parity, abort_s, a.status); };
  // wait for use number `i` of a ring of n barriers
  auto wait_ring = [&](uint64_t* bars, int n, int i) { return wait(&bars[i % n], (uint32_t)(i / n) & 1u); };
  const int shift = a.pool.shift;
  const int per_tile = kKT >> shift;
  const uint32_t all_ok = (per_tile == 32 ? 0xffffffffu : (1u << per_tile) - 1);

  // The copies of a unit's keys (kv = 0) or values (kv = 1); `c` counts key
  // tiles.  The values' warp also leaves each tile's block mask and, of an
  // 8-bit pool, the exponent bytes of keys and values, before it announces
  // the copy: the softmax waits for that one.
  auto copies = [&](const Walk<RQ, kKT>& w, int kv, int& c) -> bool {
    Feed<Q8> f(a, w.u.b, w.u.h, w.s.len, w.kt0, w.kt1);
    const int n = Q8 ? RS : kv ? VS : KS;
    for (int kt = w.kt0; kt < w.kt1; f.advance(kt), ++kt, ++c) {
      const unsigned ok = __ballot_sync(0xffffffffu, f.cur >= 0);
      const int rows = __popc(ok) << shift;
      const int64_t row = ((int64_t)f.cur * a.pool.Hkv + w.u.h) << shift;
      const int st = c % n;
      uint64_t* full = Q8 ? &raw_full[st * 2 + kv] : (kv ? vfull : kfull) + st;
      if (c >= n && !wait(Q8 ? &raw_empty[st * 2 + kv] : (kv ? vempty : kempty) + st, (uint32_t)(c / n - 1) & 1u))
        return false;
      if (kv == 1) {
        int top = 0;
        if (Q8) {
          if (lane < 16) *reinterpret_cast<uint4*>(ex_s + (c & 15) * 256 + lane * 16) = f.ex;
          top = __shfl_sync(0xffffffffu, f.largest(), 8);
        }
        if (lane == 0) info_s[c & 15] = make_uint2(ok, (uint32_t)top);
        __syncwarp();
      }
      if (lane == 0) {
        if (rows) mbar_arrive_expect(full, (uint32_t)rows * D * (Q8 ? 1 : 2));
        else mbar_arrive(full);
      }
      __syncwarp();
      if (f.cur >= 0) {
        if constexpr (Q8) {
          unsigned char* dst = sm + S::off_raw + (st * 2 + kv) * S::kRaw;
          bulk_g2s(dst + (lane << shift) * D, static_cast<const uint8_t*>(kv ? a.pool.V : a.pool.K) + row * D,
                   (uint32_t)D << shift, full);
        } else {
          const CUtensorMap* map = kv ? &maps.V : &maps.K;
          unsigned char* d = sm + (kv ? S::off_V : S::off_K) + (size_t)st * S::kTile + (lane << shift) * 128;
          tma_load_box(d, map, 0, (int)row, full);
          if (D == 128) tma_load_box(d + kHalfBytes, map, 64, (int)row, full);
        }
      }
    }
    return true;
  };
  // after a wait has given up: copies still in flight land before the CTA ends
  auto drain = [&](int kv, int c) {
    __syncwarp();
    if (!*abort_s || lane != 0) return;
    const int n = Q8 ? RS : kv ? VS : KS;
    for (int i = c - 1; i >= 0 && i >= c - n; --i)
      (void)mbar_wait(Q8 ? &raw_full[(i % n) * 2 + kv] : (kv ? vfull : kfull) + i % n, (uint32_t)(i / n) & 1u, a.status);
  };

  if (Q8 && warp < 4) regs_dec<72>();
  if (warp == 0) {
    // ============================================================== keys
    int c = 0;
    bool go = true;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) go = copies(w, 0, c);
    drain(0, c);
  } else if (warp == 1) {
    // ============================================================== S^T = K Q^T
    if (lane == 0) {
      const uint32_t idS = Q8 ? idesc_f16(128, NQ, false, false) : tc::idesc_bf16(128, NQ, false, false);
      const uint32_t qb = smem_u32(sm + S::off_Q), kb = smem_u32(sm + S::off_K);
      int c = 0, k = 0;  // key tiles, units
      bool go = true;
      for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next(), ++k) {
        if (!(go = wait_ring(q_full, 2, k))) break;
        const uint64_t qd = tc::desc_kmajor_sw128(qb + (uint32_t)(k & 1) * S::kQ);
        const int T = w.kt1 - w.kt0;
        for (int j = 0; j < T; ++j, ++c) {
          if (!(go = (c < 2 || wait_ring(s_free, 2, c - 2)) && wait_ring(kfull, KS, c))) break;
          tc::fence_after_sync();
          const uint64_t kd = tc::desc_kmajor_sw128(kb + (uint32_t)(c % KS) * S::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // (the address field of a descriptor counts 16 bytes)
            tc::mma_bf16(tmem + (c & 1) * 64, kd + (((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4),
                         qd + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idS, kk > 0);
          tc::mma_commit(&s_full[c & 1]);
          tc::mma_commit(&kempty[c % KS]);
          if (j == T - 1) tc::mma_commit(&q_empty[k & 1]);
        }
      }
      if (c > 0) {
        tc::mma_commit(&fin[0]);
        (void)mbar_wait(&fin[0], 0, a.status);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ============================================================== O^T += V^T P^T
    if (lane == 0) {
      const uint32_t idO = Q8 ? idesc_f16(128, NQ, true, false) : tc::idesc_bf16(128, NQ, true, false);
      const uint32_t pb = smem_u32(sm + S::off_P), vb = smem_u32(sm + S::off_V);
      int c = 0;
      bool go = true;
      for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) {
        const int T = w.kt1 - w.kt0;
        for (int j = 0; j < T; ++j, ++c) {
          if (!(go = wait_ring(vfull, VS, c) && wait_ring(p_ready, 2, c))) break;
          tc::fence_after_sync();
          const uint64_t vd = tc::desc_mnmajor_sw128(vb + (uint32_t)(c % VS) * S::kTile, kHalfBytes);
          const uint64_t pd = tc::desc_kmajor_sw128(pb + (uint32_t)(c & 1) * S::kP);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16(tmem + kColO, vd + kk * (2048 >> 4), pd + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idO,
                         j > 0 || kk > 0);
          tc::mma_commit(&pv_done[c & 1]);
          tc::mma_commit(&vempty[c % VS]);
        }
      }
      if (c > 0) {
        tc::mma_commit(&fin[1]);
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
  } else if (warp < 8) {
    // ============================================================== softmax
    if (Q8) regs_inc<248>();
    const int r = tid & 127;  // key of the tile; channel of O^T
    const int q4 = warp & 3;
    const uint32_t tl = (uint32_t)(32 * q4) << 16;
    constexpr int CH = RQ < 16 ? 8 : 16;  // columns of a TMEM load
    auto load_cols = [&](uint32_t at, float (&v)[CH]) {
      if constexpr (CH == 8) tc::tmem_ld8(at, v);
      else tc::tmem_ld16(at, v);
    };
    int c = 0, k = 0;
    bool go = true;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next(), ++k) {
      const int T = w.kt1 - w.kt0;
      const float* qe = qe_s + (k & 15) * NQ;
      float cv = 0.f;  // (8-bit) the unit's value exponent: sums of weights are in units of 2^cv
      const int p0 = (int)(w.s.len - w.s.n), g0 = (int)w.u.i * RQ;
      const int pos_lo = p0 + g0 / a.G, pos_hi = p0 + (g0 + w.nrow - 1) / a.G;
      auto first_of = [&](int pos) { return a.window > 0 && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0; };
      const int first_lo = first_of(pos_lo), first_hi = first_of(pos_hi);
      bar_named_sync(2, 128);  // the last unit's readers are done
      if (r < RQ) {
        const int pos = p0 + (g0 + (r < w.nrow ? r : w.nrow - 1)) / a.G;
        pos_s[r] = make_int2(first_of(pos), pos);  // the row's keys
        m_s[r] = -INFINITY;
      }
      bar_named_sync(2, 128);
      float l[RQ];
#pragma unroll
      for (int n = 0; n < RQ; ++n) l[n] = 0.f;
      for (int j = 0; j < T; ++j, ++c) {
        const int k0 = (w.kt0 + j) * kKT, t = k0 + r;
        go = __all_sync(0xffffffffu, (c < 2 || wait_ring(pv_done, 2, c - 2)) && wait_ring(vfull, VS, c) &&
                                         wait_ring(s_full, 2, c));
        // (a failed wait is carried to the barrier below, where the four warps leave together)
        const uint2 info = info_s[c & 15];
        const uint32_t ok = info.x;
        const bool masked = k0 + 127 > pos_lo || k0 < first_hi || ok != all_ok;
        const bool live = t < w.s.len && ((ok >> (r >> shift)) & 1u);
        float ks = a.scale_log2, ve = 0.f, pe = 1.f;
        if constexpr (Q8) {
          // (rows of exponent 255 hold NaN codes: any factor will do)
          const int e0 = ex_s[(c & 15) * 256 + r], e1 = ex_s[(c & 15) * 256 + 128 + r];
          if (j == 0) cv = info.y ? (float)((int)max(info.y, 7u) - 127) : 0.f;
          ks *= exp2i(e0 == 255 ? 0 : max(e0, 7) - 127);
          ve = (float)(e1 == 255 ? 0 : max(e1, 7) - 127);
          pe = exp2i(min(max((int)(cv - ve), -126), 126));
        }
        if (masked && go && (!live || t < first_lo)) {
          // no row's key: the weights' zeros must not meet what the pool
          // holds there, or what shared memory held before
          unsigned char* v = sm + S::off_V + (size_t)(c % VS) * S::kTile;
#pragma unroll
          for (int q = 0; q < D / 8; ++q)
            *reinterpret_cast<uint4*>(v + (q >> 3) * kHalfBytes + sw_off(r, q)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
        tc::fence_after_sync();
        float y[RQ];
        const uint32_t st = tmem + tl + (c & 1) * 64;
#pragma unroll
        for (int n0 = 0; n0 < RQ; n0 += CH) {
          float v[CH];
          load_cols(st + n0, v);
#pragma unroll
          for (int n = 0; n < CH; ++n) y[n0 + n] = Q8 ? fmaf(v[n], ks * qe[n0 + n], ve) : v[n] * ks;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[c & 1]);
        if (masked) {
#pragma unroll
          for (int n = 0; n < RQ; ++n) {
            const int2 fl = pos_s[n];
            y[n] = live && t >= fl.x && t <= fl.y ? y[n] : -INFINITY;
          }
        }
        bool grow = j == 0 || !go;
#pragma unroll
        for (int n = 0; n < RQ; n += 4) {
          const float4 mr = *reinterpret_cast<const float4*>(m_s + n);
          grow |= y[n] > mr.x + kTau || y[n + 1] > mr.y + kTau || y[n + 2] > mr.z + kTau || y[n + 3] > mr.w + kTau;
        }
        if (bar_red_or(1, 128, grow)) {
          go = !bar_red_or(1, 128, !go);
          if (!go) break;
          // new maxima: over the warp's keys, then over the four warps
#pragma unroll
          for (int n = 0; n < RQ; ++n) {
            const float x = warp_max(y[n]);
            if (lane == n % 32) red_s[q4 * 64 + n] = x;
          }
          bar_named_sync(2, 128);
          float f[RQ];
#pragma unroll
          for (int n = 0; n < RQ; ++n) {
            const float x = fmaxf(fmaxf(red_s[n], red_s[64 + n]), fmaxf(red_s[128 + n], red_s[192 + n]));
            const float m = m_s[n];
            f[n] = x > m ? (m == -INFINITY ? 0.f : ex2_approx(m - x)) : 1.f;
            l[n] *= f[n];
          }
          if (j > 0) {
            go = __all_sync(0xffffffffu, wait_ring(pv_done, 2, c - 1));
            if (go) {
              tc::fence_after_sync();
#pragma unroll
              for (int n0 = 0; n0 < RQ; n0 += 8) {
                float o[8];
                tc::tmem_ld8(tmem + tl + kColO + n0, o);
#pragma unroll
                for (int n = 0; n < 8; ++n) o[n] *= f[n0 + n];
                tc::tmem_st8(tmem + tl + kColO + n0, o);
              }
            }
          }
          bar_named_sync(2, 128);  // every thread has read m_s
          if (r < RQ) {
            const float x = fmaxf(fmaxf(red_s[r], red_s[64 + r]), fmaxf(red_s[128 + r], red_s[192 + r]));
            m_s[r] = fmaxf(x, m_s[r]);
          }
          if (bar_red_or(1, 128, !go)) {
            go = false;
            break;
          }
        }
        // weights
        unsigned char* P = sm + S::off_P + (size_t)(c & 1) * S::kP + (r >> 6) * NQ * 128 + (r & 7) * 2;
        const int ch = (r & 63) >> 3;
#pragma unroll
        for (int n = 0; n < RQ; n += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(m_s + n);
          const float mr[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p = ex2_approx(y[n + q] - (mr[q] == -INFINITY ? 0.f : mr[q]) + (Q8 ? kUp : 0.f));
            l[n + q] = fmaf(p, pe, l[n + q]);
            *reinterpret_cast<uint16_t*>(P + (n + q) * 128 + ((ch ^ ((n + q) & 7)) << 4)) =
                Q8 ? (uint16_t)pack_f16x2(p, 0.f) : (uint16_t)pack_bf16x2(p, 0.f);
          }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[c & 1]);
      }
      if (!go) break;
      // ---- the unit's result, or this CTA's piece of it
      go = __all_sync(0xffffffffu, wait_ring(pv_done, 2, c - 1));
      tc::fence_after_sync();
#pragma unroll
      for (int n = 0; n < RQ; ++n) {
        const float x = warp_sum(l[n]);
        if (lane == n % 32) red_s[q4 * 64 + n] = x;
      }
      if (bar_red_or(1, 128, !go)) {
        go = false;
        break;
      }
      const bool whole = w.whole();
      const int64_t at = (int64_t)w.slot(blockIdx.x) * RQ;
      // 8-bit: O^T is in units of 2^(m - kUp), the sums of 2^(m - kUp - cv)
      const float up = Q8 ? exp2i((int)cv) : 1.f, dm = Q8 ? kUp + cv : 0.f;
#pragma unroll 1
      for (int n0 = 0; n0 < RQ; n0 += 8) {
        float o[8];
        tc::tmem_ld8(tmem + tl + kColO + n0, o);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int row = n0 + n;
          if (row < w.nrow) {
            const float sum = (red_s[row] + red_s[64 + row]) + (red_s[128 + row] + red_s[192 + row]);
            const int g = g0 + row, tok = g / a.G, head = w.u.h * a.G + g % a.G;
            if (whole) {
              const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
              if (r < D)
                (static_cast<__nv_bfloat16*>(a.out) + (w.s.r0 + tok) * a.ot + (int64_t)head * a.oh)[r] =
                    __float2bfloat16_rn(o[n] * up * inv);
              if (r == 0 && a.lse)
                a.lse[(w.s.r0 + tok) * a.Hq + head] = (m_s[row] - dm + log2f(sum)) * 0.6931471805599453f;
            } else {
              if (r < D) a.part[(at + row) * D + r] = o[n] * up;
              if (r == 0) a.ml[at + row] = make_float2(m_s[row] - dm, sum);
            }
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
    }
  } else if constexpr (Q8) {
    // ============================================================== codes to bf16 tiles
    regs_dec<96>();
    int c = 0;
    bool go = true;
    const int t = tid & 127, kv = (warp - 8) >> 2;
    const int n = kv ? VS : KS;
    uint64_t* full = kv ? vfull : kfull;
    uint64_t* empty = kv ? vempty : kempty;
    for (Walk<RQ, kKT> w(a, Wb, blockIdx.x); w.more() && go; w.next()) {
      for (int j = 0; j < w.kt1 - w.kt0; ++j, ++c) {
        const int raw = (c % RS) * 2 + kv;
        go = __all_sync(0xffffffffu, wait(&raw_full[raw], (uint32_t)(c / RS) & 1u) &&
                                         (c < n || wait(&empty[c % n], (uint32_t)(c / n - 1) & 1u)));
        if (!go) break;
        const unsigned char* src = sm + S::off_raw + raw * S::kRaw;
        unsigned char* dst = sm + (kv ? S::off_V : S::off_K) + (size_t)(c % n) * S::kTile;
        convert_tile<D, false>(src, nullptr, dst, t);  // (the softmax multiplies by the powers of two)
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
  // 128 (72 + 248 + 96 + 96) = 512 * 128
  if (e == cudaSuccess && Q8) e = check_registers<pool_few_kernel<D, RQ, Q8>>(128);
  if (e == cudaSuccess && a.planned) e = launch_plan<RQ, kKT>(a, st);
  if (e != cudaSuccess) return e;
  PoolMaps none = {};
  pool_few_kernel<D, RQ, Q8><<<a.ctas, Q8 ? 512 : 256, S::bytes, st>>>(maps ? *maps : none, a);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_merge<__nv_bfloat16, D, RQ, kKT>(a, st);
}

template <int D, bool Q8>
cudaError_t launch_few_d(const PoolAttendArgs& a, const PoolMaps* maps, int TM, cudaStream_t st) {
  switch (TM) {
    case 8: return launch_few<D, 8, Q8>(a, maps, st);
    case 16: return launch_few<D, 16, Q8>(a, maps, st);
    case 32: return launch_few<D, 32, Q8>(a, maps, st);
    default: return launch_few<D, 64, Q8>(a, maps, st);
  }
}

}  // namespace

cudaError_t launch_pool_few(const PoolAttendArgs& a, const PoolMaps* maps, int TM, int bits, int d, cudaStream_t stream) {
  if (d == 64) return bits == 8 ? launch_few_d<64, true>(a, maps, TM, stream) : launch_few_d<64, false>(a, maps, TM, stream);
  return bits == 8 ? launch_few_d<128, true>(a, maps, TM, stream) : launch_few_d<128, false>(a, maps, TM, stream);
}

}  // namespace lod
