// lod_pool_attend.cu -- exact attention of new tokens over the block pool: the
// CUDA-core kernel and the choice of kernel.
#include <cuda_fp8.h>

#include "lod_pool_list.cuh"

namespace lod {
namespace {

// ---------------------------------------------------------------- CUDA cores

// fp32 attention on the CUDA cores.  A CTA of 4 * TM threads (128 at least)
// holds a tile of TM query rows; per tile of KT keys S = Q K^T and O += P V
// from shared memory, each thread RPT rows x KPT keys of S and the same rows x
// D/16 channels of O, so 16 neighbouring lanes own a row and its maximum and
// sum need no shared memory.  fp32 has no tensor-core form of its own accuracy,
// so the FMA pipe bounds it; per 4 channels a thread reads RPT + KPT vectors
// for 4 RPT KPT FMAs (as pairs: fma.rn.f32x2).
// 64 rows of 128 channels take 32 keys a tile and not 64, so that two CTAs fit
// an SM: 2 x 500 tokens over 3001, 8 / 2 heads, 410 us (27 TFLOP/s) against
// 447; with 8 rows a thread and 4 warps a CTA 567.
template <int D, int TM>
constexpr int kSimtKT = D == 128 && TM == 64 ? 32 : 64;
template <typename T, int D, int TM, bool Q8>
__global__ void __launch_bounds__(TM == 16 ? 128 : 256, 2) pool_simt_kernel(PoolAttendArgs a) {
  constexpr int KT = kSimtKT<D, TM>, KPT = KT / 16, NT = TM == 16 ? 128 : 256, RPT = TM * 16 / NT, CPT = D / 16;
  constexpr int KS = D + 4, PS = KT + 4;
  constexpr int E = 16 / (int)sizeof(T), PPR = D / E;
  static_assert(E == 4, "fp32 rows");
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;               // [TM][D]
  float* Ks = Qs + TM * D;      // [KT][KS]
  float* Vs = Ks + KT * KS;     // [KT][D]
  float* Ps = Vs + KT * D;      // [TM][PS]
  int* live = reinterpret_cast<int*>(Ps + TM * PS);  // [2][KT]: the key exists (two tiles: they are loaded ahead)
  __shared__ int64_t wb_s[kInlineSeqs + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

  const int64_t* Wb = a.Wb;
  if (a.planned) pdl_wait();  // (the plan)
  if (!a.planned) {
    plan_inline<TM, KT>(a, wb_s);
    Wb = wb_s;
  }
  clear_refused<T, D, false>(a, Wb);
  Walk<TM, KT> w(a, Wb, blockIdx.x);
  for (; w.more(); w.next()) {
    const Unit& u = w.u;
    const SeqView& s = w.s;
    const int kt0 = w.kt0, kt1 = w.kt1, nrow = w.nrow;
    const int64_t row0 = u.i * TM;
    const int32_t* table = a.batch.table + (int64_t)u.b * a.batch.max_blocks;
    // (earlier and later keys are no row's)
    const int64_t first_unit = a.window > 0 ? s.len - s.n + row0 / a.G - a.window + 1 : 0;
    const int64_t last_unit = s.len - s.n + (row0 + nrow - 1) / a.G;

    __syncthreads();
    for (int x = tid; x < TM * PPR; x += NT) {
      const int r = x / PPR, c = x % PPR;
      float v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = 0.f;
      if (r < nrow) {
        const int64_t g = row0 + r;
        const T* q = static_cast<const T*>(a.q) + (s.r0 + g / a.G) * a.qt + (u.h * a.G + g % a.G) * a.qh;
        load_f<T, E>(q + c * E, v);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) Qs[r * D + c * E + i] = v[i];
    }
    float m[RPT], l[RPT];
    float2 acc[RPT][CPT / 2];
    int64_t pos[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = ty * RPT + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
      pos[i] = r < nrow ? s.len - s.n + (row0 + r) / a.G : -1;
#pragma unroll
      for (int j = 0; j < CPT / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
    }
    // One tile's keys (z = 0) or values (z = 1) to shared memory, as fp32.
    // fp32 rows go by asynchronous copies: the next tile's keys while this
    // tile's weights meet the values, its values during the next scores.
    auto load_tile = [&](int kt, int z) {
      for (int x = tid; x < KT * PPR; x += NT) {
        const int k = x / PPR, c = x % PPR;
        const int64_t t = (int64_t)kt * KT + k;
        int64_t blk = -1;
        if (t <= last_unit && t >= first_unit) {
          blk = table[t >> a.pool.shift];
          if (blk < 0 || blk >= a.pool.blocks) {
            blk = -1;
            set_status(a.status, LOD_ST_BAD_PAGE);
          }
        }
        if (z == 0 && c == 0) live[(kt & 1) * KT + k] = blk >= 0;
        const int64_t row = ((blk * a.pool.Hkv + u.h) << a.pool.shift) + (t & (((int64_t)1 << a.pool.shift) - 1));
        const void* base = z ? a.pool.V : a.pool.K;
        float* to = z ? &Vs[k * D + c * E] : &Ks[k * KS + c * E];
        if constexpr (!Q8) {
          cp_async16_zfill(to, blk >= 0 ? static_cast<const T*>(base) + row * D + c * E : static_cast<const T*>(base),
                           blk >= 0);
        } else {
          float v[E];
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = 0.f;
          if (blk >= 0) {
            const uint8_t* src = static_cast<const uint8_t*>(base) + row * D + c * E;
            const int E8 = (z ? a.pool.Ve : a.pool.Ke)[row];
            const float f = E8 == 255 ? NAN : E8 == 0 ? __uint_as_float(0x400000u) : __uint_as_float((uint32_t)E8 << 23);
            const uint32_t word = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * j)), __NV_E4M3);
              const float2 f2 = __half22float2(__half2(hr));
              v[2 * j] = f2.x * f;
              v[2 * j + 1] = f2.y * f;
            }
          }
          *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      if constexpr (!Q8) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load_tile(kt0, 0);
    load_tile(kt0, 1);
    for (int kt = kt0; kt < kt1; ++kt) {
      // this tile's keys (the values may still be on their way)
      if constexpr (!Q8) asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      // S: rows ty * RPT + i, keys tx + 16 j, even and odd channels apart
      float sc[RPT][KPT];
      {
        float2 s2[RPT][KPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < KPT; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int e = 0; e < D; e += 4) {
          float4 kk[KPT], qq[RPT];
#pragma unroll
          for (int j = 0; j < KPT; ++j) kk[j] = *reinterpret_cast<const float4*>(&Ks[(tx + 16 * j) * KS + e]);
#pragma unroll
          for (int i = 0; i < RPT; ++i) qq[i] = *reinterpret_cast<const float4*>(&Qs[(ty * RPT + i) * D + e]);
#pragma unroll
          for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
              s2[i][j] = ffma2(make_float2(qq[i].x, qq[i].y), make_float2(kk[j].x, kk[j].y), s2[i][j]);
              s2[i][j] = ffma2(make_float2(qq[i].z, qq[i].w), make_float2(kk[j].z, kk[j].w), s2[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < KPT; ++j) sc[i][j] = s2[i][j].x + s2[i][j].y;
      }
      __syncthreads();  // the keys have been read
      if (kt + 1 < kt1) load_tile(kt + 1, 0);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
          const int k = tx + 16 * j;
          const int64_t t = (int64_t)kt * KT + k;
          const bool seen = live[(kt & 1) * KT + k] && t <= pos[i] && (a.window <= 0 || t > pos[i] - a.window);
          sc[i][j] = seen ? sc[i][j] * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, sc[i][j]);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // a row that has seen no key yet
        const float f = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
          const float p = exp2f(sc[i][j] - ref);
          sum += p;
          Ps[(ty * RPT + i) * PS + tx + 16 * j] = p;
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = fmaf(l[i], f, sum);
        m[i] = mn;
#pragma unroll
        for (int j = 0; j < CPT / 2; ++j) acc[i][j] = make_float2(acc[i][j].x * f, acc[i][j].y * f);
      }
      // this tile's values (the next keys may still be on their way)
      if constexpr (!Q8) {
        if (kt + 1 < kt1) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
#pragma unroll 2
      for (int k = 0; k < KT; k += 4) {
        float4 pp[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) pp[i] = *reinterpret_cast<const float4*>(&Ps[(ty * RPT + i) * PS + k]);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
#pragma unroll
          for (int c = 0; c < CPT / 4; ++c) {
            const float4 vv = *reinterpret_cast<const float4*>(&Vs[(k + z) * D + c * 64 + tx * 4]);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const float p = z == 0 ? pp[i].x : z == 1 ? pp[i].y : z == 2 ? pp[i].z : pp[i].w;
              acc[i][2 * c] = ffma2(make_float2(p, p), make_float2(vv.x, vv.y), acc[i][2 * c]);
              acc[i][2 * c + 1] = ffma2(make_float2(p, p), make_float2(vv.z, vv.w), acc[i][2 * c + 1]);
            }
          }
        }
      }
      __syncthreads();  // the values have been read
      if (kt + 1 < kt1) load_tile(kt + 1, 1);
    }
    // the unit's result, or this CTA's piece of it
    const bool whole = w.whole();
    const int slot = w.slot(blockIdx.x);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = ty * RPT + i;
      if (r >= nrow) continue;
      const int64_t g = row0 + r, tok = s.r0 + g / a.G, head = u.h * a.G + g % a.G;
      if (whole) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        T* o = static_cast<T*>(a.out) + tok * a.ot + head * a.oh;
#pragma unroll
        for (int c = 0; c < CPT / 4; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            o[c * 64 + tx * 4 + 2 * j] = Elem<T>::from_f(acc[i][2 * c + j].x * inv);
            o[c * 64 + tx * 4 + 2 * j + 1] = Elem<T>::from_f(acc[i][2 * c + j].y * inv);
          }
        if (tx == 0 && a.lse) a.lse[tok * a.Hq + head] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
      } else {
        float* o = a.part + ((int64_t)slot * TM + r) * D;
#pragma unroll
        for (int c = 0; c < CPT / 4; ++c)
          *reinterpret_cast<float4*>(o + c * 64 + tx * 4) =
              make_float4(acc[i][2 * c].x, acc[i][2 * c].y, acc[i][2 * c + 1].x, acc[i][2 * c + 1].y);
        if (tx == 0) a.ml[(int64_t)slot * TM + r] = make_float2(m[i], l[i]);
      }
    }
  }
  if (tid == 0) w.record(blockIdx.x);
}

template <typename T, int D, int TM, bool Q8>
cudaError_t launch_simt(const PoolAttendArgs& a, cudaStream_t st) {
  constexpr int KT = kSimtKT<D, TM>;
  constexpr size_t smem = sizeof(float) * (TM * D + KT * (D + 4) + KT * D + TM * (KT + 4)) + 2 * sizeof(int) * KT;
  cudaError_t e = set_smem_once<pool_simt_kernel<T, D, TM, Q8>>(smem);
  if (e == cudaSuccess && a.planned) e = launch_plan<TM, KT>(a, st);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.ctas), block(TM == 16 ? 128 : 256);
  if (a.planned) {
    e = launch_pdl(pool_simt_kernel<T, D, TM, Q8>, grid, block, smem, st, a);
  } else {
    pool_simt_kernel<T, D, TM, Q8><<<grid, block, smem, st>>>(a);
    e = cudaGetLastError();
  }
  return e != cudaSuccess ? e : launch_merge<T, D, TM, KT>(a, st);
}

template <typename T, int D>
cudaError_t launch_simt_d(const PoolAttendArgs& a, int TM, int bits, cudaStream_t st) {
  if (TM == 16) return bits == 8 ? launch_simt<T, D, 16, true>(a, st) : launch_simt<T, D, 16, false>(a, st);
  return bits == 8 ? launch_simt<T, D, 64, true>(a, st) : launch_simt<T, D, 64, false>(a, st);
}

}  // namespace

PoolShape pool_shape(int dtype, int bits, int d, int Hkv, int G, int B, int64_t capacity, int64_t N, int64_t max_new,
                     int sms) {
  PoolShape s = {};
  s.max_rounds = 1;
  const int64_t rows = max_new * G;
  s.kind = dtype != LOD_DTYPE_BF16 ? 0 : rows > (bits == 8 ? 32 : 64) ? 1 : 2;
  if (s.kind == 2) {
    s.TM = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    s.ctas = sms;
    s.inline_plan = B <= kInlineSeqs;
  } else if (s.kind == 1) {
    s.TM = 256;
    s.ctas = sms;
    s.inline_plan = false;
    const int64_t bytes = capacity * B * Hkv * pool_row_bytes(dtype, bits, d);
    s.max_rounds = (int)(bytes > kRoundBytes * kMaxRounds ? kMaxRounds : (bytes + kRoundBytes - 1) / kRoundBytes);
  } else {
    s.TM = max_new * G <= 16 ? 16 : 64;
    s.ctas = sms * 2;  // (two CTAs an SM)
    s.inline_plan = max_new * G <= s.TM && B <= kInlineSeqs;
  }
  const int64_t tiles = N * G / s.TM + B;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  s.off_plan = kWsHeader;
  size_t plan = s.inline_plan ? 0 : (size_t)(B + 1) * 16 + (size_t)tiles * 4 + 16;
  s.off_ml = s.off_plan + up(plan);
  s.off_rec = s.off_ml + up((size_t)s.ctas * s.max_rounds * 2 * s.TM * sizeof(float2));
  s.off_part = s.off_rec + up((size_t)s.ctas * s.max_rounds * sizeof(MergeRec));
  s.total = s.off_part + up((size_t)s.ctas * s.max_rounds * 2 * s.TM * d * sizeof(float));
  return s;
}

cudaError_t launch_pool_attend(PoolAttendArgs& a, const PoolShape& s, const PoolMaps* maps, int dtype, int bits, int d,
                               cudaStream_t stream) {
  if (s.kind == 1) return launch_pool_rows(a, maps, bits, d, stream);
  if (s.kind == 2) return launch_pool_few(a, maps, s.TM, bits, d, stream);
  return d == 64 ? launch_simt_d<float, 64>(a, s.TM, bits, stream) : launch_simt_d<float, 128>(a, s.TM, bits, stream);
}

}  // namespace lod
