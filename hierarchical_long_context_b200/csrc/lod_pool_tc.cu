// lod_pool_tc.cu -- exact attention of many new tokens over the block pool on the
// tensor cores (tcgen05, TMEM accumulators, TMA): 256 query rows per unit.
#include <cfloat>

#include "lod_pool_list.cuh"
#include "lod_pool_tc.cuh"

namespace lod {
namespace {

constexpr int kTM = 256;  // query rows of a unit

// ---------------------------------------------------------------- kernel

template <int D, bool Q8>
struct RowsSmem {
  static constexpr int kTile = 128 * D * 2;  // a K, V or Q tile
  static constexpr int kStages = D == 128 ? (Q8 ? 4 : 5) : 8;
  static constexpr int kRaw = Q8 ? 128 * D + 128 + 256 : 0;  // codes, exponent bytes and row factors of a tile
  static constexpr size_t off_Q = 0;                   // two query tiles
  static constexpr size_t off_KV = off_Q + 2 * kTile;  // ring: K, V of a key tile take turns
  static constexpr size_t off_raw = off_KV + (size_t)kStages * kTile;
  static constexpr size_t off_bar = off_raw + 2 * kRaw;
  static constexpr int kBars = 2 * kStages + 6 + 4 + 4 + 2 + 2 + 2 + 2;
  static constexpr size_t off_info = off_bar + 8 * kBars + 8;  // int [2][16] a tile's largest exponents, [2][16] its blocks
  static constexpr size_t bytes = off_info + 256 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
};

// Roles: warp 0 copies, warps 1 and 2 the MMAs of query tiles 0 and 1 (one
// issuer for both took 1000 cycles a step of 512 to 640 cycles' work); warps 4-7
// and 8-11 the softmax of query tiles 0 and 1 (a thread per row); with an
// 8-bit pool warps 12-15 turn codes into f16 tiles and warp 3 their exponents
// into factors.  Such a tile's rows are taken relative to its largest exponent, C: the keys' 2^C
// joins the softmax scale, the values' joins the weights' exponent, and O_s
// is kept in units of a running largest C.
//
// Tensor memory: S_0, S_1 (fp32, 128 columns each; the weights P_s, bf16
// pairs, overwrite the first half of each 64-column half of S_s), O_0, O_1.
// Scores, weights and sums go by halves of 64 keys: for each half u the
// issuer of query tile s gives O_s += P_s V_j (half u), then S_s = Q_s
// K_{j+1}^T (half u), so a softmax warpgroup works on one half while the
// MMAs of its other half run.  (With one buffer of 128 keys a warpgroup waited
// 1550 of every 3650 cycles for its own MMAs.)
// The softmax warps rescale O_s themselves, and only when a row's maximum has
// grown by more than 2^8 (weights up to 2^8 are as exact as any in bf16 and
// fp32).
// Bounds, per 128 keys and 256 rows: 2048 cycles of tensor work (d = 128; 2560
// with the scores' MMAs of 64 keys, which read their queries twice as often),
// 2048 of exponentials on the special-function unit alone (16 a clock).
// Measured: 2048 new tokens over 128K, 32 / 8 heads, 4.30 ms (1.0 PFLOP/s) in a
// loop, where the power cap holds the clock at 1.45 GHz, 3.8 ms before it does.
template <int D, bool Q8>
__global__ void __launch_bounds__(Q8 ? 512 : 384, 1)
    pool_rows_kernel(const __grid_constant__ PoolMaps maps, const __grid_constant__ PoolAttendArgs a) {
  using S = RowsSmem<D, Q8>;
  constexpr int NS = S::kStages;
  constexpr float kTau = 8.f;
  constexpr float kUp = 6.f;  // 8-bit: weights are up to 2^15 of f16's 2^16
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::off_bar);
  uint64_t* empty = full + NS;
  uint64_t* raw_full = empty + NS;
  uint64_t* raw_empty = raw_full + 2;
  uint64_t* fac_full = raw_empty + 2;
  uint64_t* s_full = fac_full + 2;
  uint64_t* p_ready = s_full + 4;  // (of query tile and key half: [2][2])
  uint64_t* q_full = p_ready + 4;
  uint64_t* pv_done = q_full + 2;
  uint64_t* o_full = pv_done + 2;
  uint64_t* fin = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 2);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* info_s = reinterpret_cast<int*>(sm + S::off_info);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], Q8 ? 4 : 1);
      mbar_init(&empty[i], 2);  // one of each query tile
    }
    for (int i = 0; i < 2; ++i) {  // (keys', values')
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
      mbar_init(&fac_full[i], 1);
      mbar_init(&q_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&fin[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
    }
    *abort_s = 0;
    fence_mbar_init();
    if (!Q8) {
      tc::prefetch_tensormap(&maps.K);
      tc::prefetch_tensormap(&maps.V);
    }
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
  pdl_wait();               // (the plan)
  clear_refused<__nv_bfloat16, D, true>(a, a.Wb);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColO = 256;

  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_or_abort(bar, parity, abort_s, a.status); };
  const int shift = a.pool.shift, parts = list_parts(a);
  const int per_tile = kKT >> shift;  // blocks of a key tile

  if (warp < 4) {
    regs_dec<Q8 ? 80 : 104>();
    if (warp == 0) {
      // ============================================================ copies
      int t = 0;  // key tiles; the ring takes their keys and values in turn
      bool go = true;
      for (int part = blockIdx.x; part < parts && go; part += a.ctas)
      for (Walk<kTM, kKT> w(a, a.Wb, part); w.more() && go; w.next()) {
        Feed f(a, w.u.b, w.s.len, w.kt0, w.kt1);
        const int Hkv = a.pool.Hkv, h = w.u.h;
        for (int kt = w.kt0; kt < w.kt1 && go; f.advance(), ++kt, ++t) {
          const unsigned ok = __ballot_sync(0xffffffffu, f.cur >= 0);
          const int rows = __popc(ok) << shift;
          const int row = (f.cur * Hkv + h) << shift;  // (a pool has fewer than 2^31 rows)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if constexpr (Q8) {
              if (t >= 1 && !(go = wait(&raw_empty[kv], (uint32_t)(t - 1) & 1u))) break;
              unsigned char* dst = sm + S::off_raw + kv * S::kRaw;
              if (lane == 0) {
                info_s[32 + kv * 16 + (t & 15)] = (int)ok;
                if (rows) mbar_arrive_expect(&raw_full[kv], (uint32_t)rows * (D + 1));
                else mbar_arrive(&raw_full[kv]);
              }
              __syncwarp();
              if (f.cur >= 0) {
                const uint8_t* codes = static_cast<const uint8_t*>(kv ? a.pool.V : a.pool.K);
                bulk_g2s(dst + (lane << shift) * D, codes + (int64_t)row * D, (uint32_t)D << shift, &raw_full[kv]);
                bulk_g2s(dst + 128 * D + (lane << shift), (kv ? a.pool.Ve : a.pool.Ke) + row, 1u << shift, &raw_full[kv]);
              }
            } else {
              const int c = 2 * t + kv, st = c % NS;
              if (c >= NS && !(go = wait(&empty[st], (uint32_t)(c / NS - 1) & 1u))) break;
              unsigned char* d = sm + S::off_KV + (size_t)st * S::kTile + (lane << shift) * 128;
              if (lane == 0) {
                if (rows) mbar_arrive_expect(&full[st], (uint32_t)rows * D * 2);
                else mbar_arrive(&full[st]);
              }
              __syncwarp();
              if (f.cur >= 0) {
                const CUtensorMap* map = kv ? &maps.V : &maps.K;
                tma_load_box(d, map, 0, row, &full[st]);
                if (D == 128) tma_load_box(d + kHalfBytes, map, 64, row, &full[st]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (*abort_s && lane == 0) {  // copies still in flight land before the CTA ends
        // (t counts a tile of which only the keys may have been asked for:
        // the wait for its values then runs out)
        for (int i = t - 1; i >= 0 && i >= t - (Q8 ? 1 : NS); --i)
          for (int kv = 0; kv < 2; ++kv)
            (void)mbar_wait(Q8 ? &raw_full[kv] : &full[(2 * i + kv) % NS], (uint32_t)(Q8 ? i : (2 * i + kv) / NS) & 1u,
                            a.status);
      }
    } else if (warp < 3) {
      // ============================================================ MMA issue, query tile s
      const int s = warp - 1;
      const uint32_t lead = elect_one();
      const uint32_t idS = Q8 ? idesc_f16(128, 64, false, false) : tc::idesc_bf16(128, 64, false, false);
      const uint32_t idO = Q8 ? idesc_f16(128, D, false, true) : tc::idesc_bf16(128, D, false, true);
      const uint32_t kvb = smem_u32(sm + S::off_KV);
      const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(sm + S::off_Q) + s * S::kTile);
      const uint64_t kd0 = tc::desc_kmajor_sw128(kvb), vd0 = tc::desc_mnmajor_sw128(kvb, kHalfBytes);
      const uint32_t ts = tmem + s * 128, to = tmem + kColO + s * 128;
      int c = 0;                 // ring position of the next K tile (V follows it)
      uint32_t np = 0, nq = 0;   // weights (of key tiles) and query tiles taken
      bool go = true, any = false;
      auto uniform = [&](bool x) { return (bool)__all_sync(0xffffffffu, x); };
      auto full_wait = [&](int x) { return uniform(wait(&full[x % NS], (uint32_t)(x / NS) & 1u)); };
      auto scores = [&](int u, int x) {  // S_s, half u: Q_s K^T, K at ring position x
        const uint64_t kd = kd0 + ((uint32_t)(x % NS) * (S::kTile >> 4) + u * (64 * 128 >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {  // (the address field of a descriptor counts 16 bytes)
          const uint32_t o = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
          mma_ss(lead, ts + u * 64, qd + o, kd + o, idS, kk > 0);
        }
        mma_commit_if(lead, &s_full[2 * s + u]);
        any = true;
      };
      int part = blockIdx.x;
      for (; part < parts && go; part += a.ctas) {
        Walk<kTM, kKT> w(a, a.Wb, part);
        for (; w.more() && go; w.next()) {
        const int T = w.kt1 - w.kt0;
        if (s * 128 >= w.nrow) {  // no second query tile: its share of the ring is given back as it fills
          for (int j = 0; j < 2 * T && go; ++j, ++c) {
            go = full_wait(c);
            if (go && lane == 0) mbar_arrive(&empty[c % NS]);
          }
          continue;
        }
        if (!(go = uniform(wait(&q_full[s], nq++ & 1u)) && full_wait(c))) break;
        tc::fence_after_sync();
        scores(0, c);
        scores(1, c);
        mma_commit_if(lead, &empty[c % NS]);
        for (int j = 0; j < T && go; ++j, ++np, c += 2) {
          const uint64_t vd = vd0 + (uint32_t)((c + 1) % NS) * (S::kTile >> 4);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            go = uniform(wait(&p_ready[2 * s + u], np & 1u)) && (u == 1 || full_wait(c + 1));
            if (!go) break;
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(lead, to, ts + u * 64 + 8 * kk, vd + (4 * u + kk) * (2048 >> 4), idO, j > 0 || u + kk > 0);
            mma_commit_if(lead, &pv_done[s]);
            if (u == 1) mma_commit_if(lead, &empty[(c + 1) % NS]);
            if (j + 1 < T) {
              if (u == 0) {
                if (!(go = full_wait(c + 2))) break;
                tc::fence_after_sync();
              }
              scores(u, c + 2);
              if (u == 1) mma_commit_if(lead, &empty[(c + 2) % NS]);
            } else if (u == 1) {
              mma_commit_if(lead, &o_full[s]);
            }
          }
        }
      }
        if (s == 0 && lane == 0) w.record(part);
      }
      // (the parts a timed-out CTA leaves: the merge must not take what an
      // earlier call recorded there, rows of another batch)
      for (; part < parts && s == 0; part += a.ctas)
        if (lane == 0) a.rec[part] = {0, 0, 0, 0, 0};
      if (any) {
        mma_commit_if(lead, &fin[s]);
        (void)mbar_wait(&fin[s], 0, a.status);
      }
      __syncwarp();
    } else if (Q8) {
      // ============================================================ row factors
      int t = 0;
      bool go = true;
      for (int part = blockIdx.x; part < parts && go; part += a.ctas)
      for (Walk<kTM, kKT> w(a, a.Wb, part); w.more() && go; w.next()) {
        // (of the keys that some row of the unit sees: what else the tile holds
        // is masked, and cleared where it is values)
        const int p0 = (int)(w.s.len - w.s.n), last_unit = p0 + ((int)w.u.i * kTM + w.nrow - 1) / a.G;
        const int64_t first_unit = a.window > 0 ? p0 + (int)w.u.i * kTM / a.G - a.window + 1 : 0;
        for (int kt = w.kt0; kt < w.kt1 && go; ++kt, ++t) {
          for (int kv = 0; kv < 2; ++kv) {
            if (!(go = __all_sync(0xffffffffu, wait(&raw_full[kv], (uint32_t)t & 1u)))) break;
            unsigned char* ex = sm + S::off_raw + kv * S::kRaw + 128 * D;
            const uint32_t e4 = reinterpret_cast<const uint32_t*>(ex)[lane];
            const int n = last_unit + 1 - kt * kKT - 4 * lane;  // tokens of this lane's four
            const int before = first_unit > 0 ? (int)first_unit - kt * kKT - 4 * lane : 0;
            const bool there = (info_s[32 + kv * 16 + (t & 15)] >> (4 * lane >> shift)) & 1;
            uint32_t live = e4 & ~__vcmpeq4(e4, 0xffffffffu);  // (a row of NaN does not count)
            live &= !there || n <= 0 ? 0u : n >= 4 ? 0xffffffffu : (1u << (8 * n)) - 1;
            live &= before <= 0 ? 0xffffffffu : before >= 4 ? 0u : 0xffffffffu << (8 * before);
            uint32_t m = __vmaxu4(live, live >> 16);
            m = __vmaxu4(m, m >> 8) & 0xff;
            const int top = (int)__reduce_max_sync(0xffffffffu, m);
            uint32_t x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              x[i] = row_factor((e4 >> (16 * i)) & 0xff, top) | row_factor((e4 >> (16 * i + 8)) & 0xff, top) << 16;
            reinterpret_cast<uint2*>(ex + 128)[lane] = make_uint2(x[0], x[1]);
            if (lane == 0) info_s[kv * 16 + (t & 15)] = top;
            __syncwarp();
            if (lane == 0) mbar_arrive(&fac_full[kv]);
          }
        }
      }
    }
  } else if (warp < 12) {
    // ============================================================== softmax
    regs_inc<Q8 ? 176 : 200>();
    const int s = (warp - 4) >> 2;  // query tile
    const int r = tid & 127;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + tl + s * 128, to = tmem + tl + kColO + s * 128;
    unsigned char* Qs = sm + S::off_Q + s * S::kTile;
    uint32_t ns = 0, no = 0;  // key halves and outputs taken
    int c = 0;                // ring position of the next key tile's K
    bool go = true;
    for (int part = blockIdx.x; part < parts && go; part += a.ctas)
      for (Walk<kTM, kKT> w(a, a.Wb, part); w.more() && go; w.next()) {
      const int T = w.kt1 - w.kt0;
      if (s * 128 >= w.nrow) {
        c += 2 * T;
        continue;
      }
      const int G = a.G, last = min(w.nrow - 1 - s * 128, 127);
      const bool mine = r <= last;
      const int g = (int)w.u.i * kTM + s * 128 + (mine ? r : last);  // (a row past the end does as the last one)
      const int tok = g / G, head = w.u.h * G + g % G;
      const int p0 = (int)(w.s.len - w.s.n);
      const int pos = p0 + tok;
      int eq = 0;  // (8-bit) the query row's power of two
      {
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(a.q) + (w.s.r0 + tok) * a.qt + (int64_t)head * a.qh;
        uint4 x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = mine ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
        if (Q8) eq = query_f16<D>(x);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4*>(Qs + (i >> 3) * kHalfBytes + sw_off(r, i)) = x[i];
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[s]);
      }
      // positions of the tile's first and last row; a bad block anywhere in
      // the piece sends its tiles through the masks
      const int pos_lo = p0 + ((int)w.u.i * kTM + s * 128) / G, pos_hi = p0 + ((int)w.u.i * kTM + s * 128 + last) / G;
      const int32_t* table = a.batch.table + (int64_t)w.u.b * a.batch.max_blocks;
      const int nblk = (int)((w.s.len + (1 << shift) - 1) >> shift);
      bool bad = false;
      for (int i = w.kt0 * per_tile + r; i < nblk && i < w.kt1 * per_tile; i += 128)
        bad |= table[i] < 0 || table[i] >= a.pool.blocks;
      const bool unit_bad = bar_red_or(1 + s, 128, bad);
      const int first = a.window > 0 && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0;  // this row's keys
      const int first_hi = a.window > 0 && pos_hi - a.window + 1 > 0 ? (int)(pos_hi - a.window + 1) : 0;

      // keys of no row of the unit's two tiles: before first_unit, behind last_unit
      const int u0 = p0 + (int)w.u.i * kTM / G, last_unit = p0 + ((int)w.u.i * kTM + w.nrow - 1) / G;
      const int first_unit = a.window > 0 && u0 - a.window + 1 > 0 ? (int)(u0 - a.window + 1) : 0;

      float m = -INFINITY, l = 0.f;
      int cv = 0, cm = 0;  // (8-bit) O_s is in units of 2^(cv - 127 - kUp); the largest tile exponent so far
      for (int j = 0; j < T && go; ++j, c += 2) {
        const int kt = w.kt0 + j;
        float scl = a.scale_log2;
        int df = 0;      // (8-bit) this tile's value exponent above cv
        float fv = 1.f;  // and the factor O_s takes for a new cv
        const bool ragged = kt * kKT + 127 > last_unit || kt * kKT < first_unit || unit_bad;  // V rows that are no keys
        if (Q8 || ragged) {
          // The tile's values (8-bit: with them its exponents).  A barrier's
          // parity tells a phase only from the one before it: the scores are
          // waited for first, as with K_j every earlier copy has landed.
          go = __all_sync(0xffffffffu, wait(&s_full[2 * s], (ns >> 1) & 1u) &&
                                           wait(&full[(c + 1) % NS], (uint32_t)((c + 1) / NS) & 1u));
          if (!go) break;
        }
        if constexpr (Q8) {
          const int ck = info_s[(c >> 1) & 15], e = max(info_s[16 + ((c >> 1) & 15)], 7);
          // the powers of two are joined first, and the factor stays in fp32's
          // normal range: 0 or infinity times a masked or zero score is NaN
          // (scores off by that are below 2^-90)
          scl *= exp2i(min(max(eq + max(ck, 7) - 127, -126), 127));
          scl = fminf(fmaxf(scl, FLT_MIN), FLT_MAX);
          // The unit of O_s follows the tiles up, and down where their values
          // are much smaller: a weight carries 2^(e - cv), and f16 drops what
          // lies 2^-30 below the largest.  It stays within 2^60 of the
          // largest, so that O_s (at most 2^44 of its unit) stays in fp32;
          // tiles of zeros leave it where it is.
          if (j == 0) cv = cm = e;
          cm = max(cm, e);
          if (e > cv + 1 || (e < cv - 8 && e > 7)) {
            const int to = max(e, cm - 60);
            fv = exp2i(max(cv - to, -126));
            cv = to;
          }
          df = max(e - cv, -60);
        }
        if (ragged) {
          // P's zeros must not meet what the pool holds behind every row's
          // position or before every row's window, or what shared memory held
          // before: those V rows become zero
          const int t = kt * kKT + r, i = t >> shift;
          if (t > last_unit || t < first_unit || table[i] < 0 || table[i] >= a.pool.blocks) {
            unsigned char* v = sm + S::off_KV + (size_t)((c + 1) % NS) * S::kTile;
#pragma unroll
            for (int q = 0; q < D / 8; ++q)
              *reinterpret_cast<uint4*>(v + (q >> 3) * kHalfBytes + sw_off(r, q)) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async();
          __syncwarp();
        }
#pragma unroll 1
        for (int u = 0; u < 2; ++u, ++ns) {
          const int k0 = kt * kKT + u * 64;
          const bool masked = k0 + 63 > pos_lo || k0 < first_hi || unit_bad;
          go = __all_sync(0xffffffffu, wait(&s_full[2 * s + u], (ns >> 1) & 1u));
          if (!go) break;
          tc::fence_after_sync();
          float y[64];
          tc::tmem_ld32xN<2>(ts + u * 64, y);
          if (masked) {
            const int hi = pos - k0, lo = first - k0;
#pragma unroll
            for (int e = 0; e < 64; ++e) y[e] = e <= hi && e >= lo ? y[e] : -INFINITY;
            if (unit_bad) {
              for (int t = k0; t < k0 + 64; t += 16) {  // (blocks are multiples of 16 tokens)
                const int i = t >> shift;
                if (i < nblk && table[i] >= 0 && table[i] < a.pool.blocks) continue;
#pragma unroll
                for (int e = 0; e < 64; ++e)
                  if (e >> 4 == (t - k0) >> 4) y[e] = -INFINITY;
              }
            }
          }
          float mx[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
          for (int e = 4; e < 60; e += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], y[e + q], y[e + 4 + q]);
          }
          float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], y[60]);
          top = max3(max3(top, y[61], y[62]), y[63], y[63]) * scl;
          // a NaN score, or an infinite one (inf - inf): the row's results are
          // NaN, whatever its weights become
          if (!(top < INFINITY)) l = NAN;
          const bool start = j == 0 && u == 0;
          const bool need = top > m + kTau || start;
          if (__any_sync(0xffffffffu, need || (fv != 1.f && u == 0))) {
            const float mn = need ? fmaxf(top, m) : m;  // (drops a NaN)
            const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
            m = mn;
            l *= f;
            const float fo = u == 0 ? f * fv : f;
            if (!start) {  // O_s, once the half before this one is in it
              go = __all_sync(0xffffffffu, wait(&pv_done[s], (ns - 1) & 1u));
              if (!go) break;
              tc::fence_after_sync();
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float o[32];
                tc::tmem_ld32(to + 32 * q, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= fo;
                tc::tmem_st32(to + 32 * q, o);
              }
            }
          }
          const float2 sc2 = make_float2(scl, scl);
          const float mu = (m == -INFINITY ? 0.f : m) - (Q8 ? (float)df + kUp : 0.f);
          const float2 mu2 = make_float2(-mu, -mu);
          float2 la[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) la[q] = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 t = ffma2(make_float2(y[32 * q + 2 * e], y[32 * q + 2 * e + 1]), sc2, mu2);
              // the exponentials are shared out between the special-function
              // unit and the FMA pipe (2 of 8 there: 2048 tokens over 128K
              // 4.29 ms, the mixed 8-bit batch of nine sequences 72.0 us; 3 of
              // 8 4.34 and 73.4, 1 of 8 4.33 and 72.5)
              if (e % 8 == 2 || e % 8 == 6) {
                t = exp2_fma2(t);
              } else {
                t.x = ex2_approx(t.x);
                t.y = ex2_approx(t.y);
              }
              la[e & 3] = fadd2(la[e & 3], t);
              pw[e] = Q8 ? pack_f16x2(t.x, t.y) : pack_bf16x2(t.x, t.y);
            }
            tmem_st16(ts + u * 64 + 16 * q, pw);
          }
          tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * s + u]);
          const float2 l2 = fadd2(fadd2(la[0], la[1]), fadd2(la[2], la[3]));
          l += (l2.x + l2.y) * (Q8 ? exp2i(-df - (int)kUp) : 1.f);
        }
      }
      // ---- the rows' results
      if (go) go = __all_sync(0xffffffffu, wait(&o_full[s], no++ & 1u));
      if (go) {
        tc::fence_after_sync();
        const bool whole = w.whole();
        const float unit = Q8 ? exp2i(cv - 127 - (int)kUp) : 1.f;
        const float inv = l > 0.f || l != l ? unit / l : 0.f;
        const int64_t at = (int64_t)w.slot(part) * kTM + s * 128 + r;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (w.s.r0 + tok) * a.ot + (int64_t)head * a.oh;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          tc::tmem_ld32(to + 32 * q, o);
          if (mine && whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4*>(out)[4 * q + e] =
                  make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                             pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                             pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<float4*>(a.part + at * D)[8 * q + e] =
                  make_float4(o[4 * e] * unit, o[4 * e + 1] * unit, o[4 * e + 2] * unit, o[4 * e + 3] * unit);
          }
          __syncwarp();
        }
        if (mine) {
          if (!whole) a.ml[at] = make_float2(m, l);
          else if (a.lse) a.lse[(w.s.r0 + tok) * a.Hq + head] = (m + log2f(l)) * 0.6931471805599453f;
        }
        tc::fence_before_sync();  // O_s is read before the next unit's weights are announced
      }
      __syncwarp();
      // a wait that gave up is one warp's own: the four leave together, as the
      // next unit opens with a barrier of theirs, which has no limit
      go = !bar_red_or(1 + s, 128, !go);
    }
  } else if constexpr (Q8) {
    // ============================================================== codes to f16 tiles
    regs_dec<80>();
    int c = 0;
    bool go = true;
    for (int part = blockIdx.x; part < parts && go; part += a.ctas)
      for (Walk<kTM, kKT> w(a, a.Wb, part); w.more() && go; w.next()) {
      for (int x = 0; x < 2 * (w.kt1 - w.kt0); ++x, ++c) {
        go = __all_sync(0xffffffffu, wait(&fac_full[c & 1], (uint32_t)(c >> 1) & 1u) &&
                                         (c < NS || wait(&empty[c % NS], (uint32_t)(c / NS - 1) & 1u)));
        if (!go) break;
        const unsigned char* src = sm + S::off_raw + (c & 1) * S::kRaw;
        convert_tile<D, true>(src, reinterpret_cast<const uint16_t*>(src + 128 * D + 128),
                              sm + S::off_KV + (size_t)(c % NS) * S::kTile, tid & 127);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[c & 1]);
          mbar_arrive(&full[c % NS]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool Q8>
cudaError_t launch_rows(const PoolAttendArgs& a, const PoolMaps* maps, cudaStream_t st) {
  cudaError_t e = set_smem_once<pool_rows_kernel<D, Q8>>(RowsSmem<D, Q8>::bytes);
  // 128 (104 + 200 + 200) = 384 * 168 and 128 (80 + 176 + 176 + 80) = 512 * 128
  if (e == cudaSuccess) e = check_registers<pool_rows_kernel<D, Q8>>(Q8 ? 128 : 168);
  if (e == cudaSuccess) e = launch_plan<kTM, kKT>(a, st);
  if (e != cudaSuccess) return e;
  PoolMaps none = {};
  e = launch_pdl(pool_rows_kernel<D, Q8>, dim3(a.ctas), dim3(Q8 ? 512 : 384), RowsSmem<D, Q8>::bytes, st, maps ? *maps : none, a);
  return e != cudaSuccess ? e : launch_merge<__nv_bfloat16, D, kTM, kKT>(a, st);
}

}  // namespace

cudaError_t launch_pool_rows(const PoolAttendArgs& a, const PoolMaps* maps, int bits, int d, cudaStream_t stream) {
  if (d == 64) return bits == 8 ? launch_rows<64, true>(a, maps, stream) : launch_rows<64, false>(a, maps, stream);
  return bits == 8 ? launch_rows<128, true>(a, maps, stream) : launch_rows<128, false>(a, maps, stream);
}

}  // namespace lod
