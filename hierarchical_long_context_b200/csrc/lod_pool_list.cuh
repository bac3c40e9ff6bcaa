// lod_pool_list.cuh -- kernels around every attention kernel of the block pool:
// the prefix sums of its work list and the merge of the units' pieces.
#pragma once

#include "lod_pool.cuh"

namespace lod {
namespace {

// ---------------------------------------------------------------- work list

// Inclusive scan of one value per thread over the CTA (1024 threads), of sums
// or of maxima; `total` receives that of all.
template <bool kMax>
__device__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto join = [](int64_t x, int64_t y) { return !kMax ? x + y : x > y ? x : y; };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = join(v, x);
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = join(s, x);
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (w > 0) v = join(v, warp_sums[w - 1]);
  *total = warp_sums[31];
  __syncthreads();
  return v;
}

// Prefix sums of the work list, for sequences with several row tiles: one CTA,
// a warp per sequence for the sums inside it.
template <int TM, int KT>
__global__ void __launch_bounds__(1024) pool_plan_kernel(PoolAttendArgs a) {
  pdl_launch_dependents();
  __shared__ int64_t ws[32];
  const int B = a.batch.B, lane = threadIdx.x & 31;
  int64_t at = 0, total, top = INT64_MIN;
  bool fell = false;  // (as in plan_inline)
  for (int b0 = 0; b0 < B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0, r0 = INT64_MIN;
    bool falls = false;
    if (b < B) {
      const SeqView q = seq_view(a.batch, a.pool.shift, b);
      n = ((int64_t)q.n * a.G + TM - 1) / TM;
      r0 = q.r0;
      falls = q.r1 < q.r0;
    }
    fell |= __syncthreads_or(falls) != 0;
    if (fell) {
      if (r0 < block_scan<true>(r0 > top ? r0 : top, ws, &total)) n = 0;
      top = total;
    }
    const int64_t s = block_scan<false>(n, ws, &total);
    if (b < B) a.RT[b + 1] = (int32_t)(at + s);
    at += total;
  }
  if (threadIdx.x == 0) a.RT[0] = 0;
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < B; b += 32) {
    const SeqView s = seq_view(a.batch, a.pool.shift, b);
    const int64_t rt = a.RT[b];
    const int64_t nt = a.RT[b + 1] - rt;
    int64_t sum = 0;
    for (int64_t i0 = 0; i0 < nt; i0 += 32) {
      const int64_t i = i0 + lane;
      int64_t n = 0;
      if (i < nt) {
        int lo, hi;
        row_tile_keys<TM, KT>(s, a.G, a.window, i, lo, hi);
        n = hi - lo + kUnitCost;
      }
      int64_t v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (i < nt) a.pre[rt + i] = (int32_t)(sum + v - n);
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) a.Wb[b + 1] = sum * a.pool.Hkv;
  }
  __syncthreads();
  at = 0;
  for (int b0 = 0; b0 < B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int64_t s = block_scan<false>(b < B ? a.Wb[b + 1] : 0, ws, &total);
    if (b < B) a.Wb[b + 1] = at + s;
    at += total;
  }
  if (threadIdx.x == 0) a.Wb[0] = 0;
  if (a.rounds) {
    int64_t keys = 0;
    for (int b0 = 0; b0 < B; b0 += 1024) {
      const int b = b0 + threadIdx.x;
      int64_t n = 0;
      if (b < B && a.RT[b + 1] > a.RT[b]) {
        const SeqView s = seq_view(a.batch, a.pool.shift, b);
        n = a.window > 0 && s.len - s.n > a.window ? a.window + s.n : s.len;
      }
      block_scan<false>(n, ws, &total);
      keys += total;
    }
    if (threadIdx.x == 0) {
      const int64_t r = (keys * a.pool.Hkv * a.row_bytes + kRoundBytes - 1) / kRoundBytes;
      // (never rounds of fewer than 64 tiles a CTA)
      const int64_t most = a.Wb[B] / ((int64_t)a.ctas * 64);
      int64_t n = r < most ? r : most;
      if (n > a.max_rounds) n = a.max_rounds;
      *a.rounds = n < 1 ? 1 : (int32_t)n;
    }
  }
}

// ---------------------------------------------------------------- merge

// Joins the pieces of the unit whose first tile lies in part c of the list and
// whose last lies behind it (there is at most one): pieces 2c + 1, 2(c + 1),
// 2(c + 2), ..., summed in a fixed order, so the result does not depend on
// which CTA ran when.  A CTA of 8 warps takes RB rows (blockIdx.y), 8 / RB
// warps to a row that share its pieces (RB = 2), or two rows to a warp (16): a
// unit of few rows is cut into many pieces, whose loads would follow one
// another in a single warp (64 pieces of one row: 10 us).
template <typename T, int D, int TM, int KT>
__global__ void __launch_bounds__(256) pool_merge_kernel(PoolAttendArgs a) {
  constexpr int RB = TM <= 16 ? 2 : 16, WPR = RB == 2 ? 4 : 1, C = D / 32;
  __shared__ float sum_s[RB == 2 ? 8 : 1][D + 1];
  pdl_wait();
  if ((int)blockIdx.x >= list_parts(a)) return;
  const MergeRec u = a.rec[blockIdx.x];
  const int nrow = u.nrow, pieces = u.pieces;
  if (pieces == 0 || (int)blockIdx.y * RB >= nrow) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % WPR;
  auto slot = [&](int i) -> int64_t { return 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0); };
#pragma unroll 1
  for (int k = warp / WPR; k < RB; k += 8 / WPR) {
    const int r = blockIdx.y * RB + k;
    if (RB != 2 && r >= nrow) break;  // (with RB = 2 every warp comes to the barriers)
    const bool live = r < nrow;
    float m = -INFINITY;
    for (int i = lane; live && i < pieces; i += 32) m = fmaxf(m, a.ml[slot(i) * TM + r].x);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[C];
#pragma unroll
    for (int j = 0; j < C; ++j) o[j] = 0.f;
#pragma unroll 4
    for (int i = slice; live && i < pieces; i += WPR) {
      const int64_t at = slot(i) * TM + r;
      const float2 x = a.ml[at];
      const float f = exp2f(x.x - ref);
      l = fmaf(x.y, f, l);
      const float* p = a.part + at * D + lane * C;
      float v[C];
      if constexpr (C == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
      } else {
        const float2 w = *reinterpret_cast<const float2*>(p);
        v[0] = w.x, v[1] = w.y;
      }
#pragma unroll
      for (int j = 0; j < C; ++j) o[j] = fmaf(v[j], f, o[j]);
    }
    if constexpr (WPR > 1) {
#pragma unroll
      for (int j = 0; j < C; ++j) sum_s[warp][lane * C + j] = o[j];
      if (lane == 0) sum_s[warp][D] = l;
      __syncthreads();
      if (slice != 0 || !live) continue;
      for (int q = 1; q < WPR; ++q) {
#pragma unroll
        for (int j = 0; j < C; ++j) o[j] += sum_s[warp + q][lane * C + j];
        l += sum_s[warp + q][D];
      }
    }
    const int g = u.g0 + r, head = u.head0 + g % a.G;
    const int64_t tok = u.r0 + g / a.G;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    T* out = static_cast<T*>(a.out) + tok * a.ot + head * a.oh + lane * C;
#pragma unroll
    for (int j = 0; j < C; ++j) out[j] = Elem<T>::from_f(o[j] * inv);
    if (lane == 0 && a.lse) a.lse[tok * a.Hq + head] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <int TM, int KT>
cudaError_t launch_plan(const PoolAttendArgs& a, cudaStream_t st) {
  pool_plan_kernel<TM, KT><<<1, 1024, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D, int TM, int KT>
cudaError_t launch_merge(const PoolAttendArgs& a, cudaStream_t st) {
  return launch_pdl(pool_merge_kernel<T, D, TM, KT>, dim3(a.ctas * a.max_rounds, TM <= 16 ? TM / 2 : TM / 16), dim3(256),
                    0, st, a);
}

}  // namespace
}  // namespace lod
