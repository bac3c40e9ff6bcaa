// lod_append.cu -- new tokens' projections into a cache (per-head norm, position
// rotation, 8-bit quantisation in the pass that stores them) and the block
// pool's read-back into a dense cache.
#include <cuda_fp8.h>

#include "lod_pool.cuh"

namespace lod {
namespace {

constexpr int kMaxPairs = 64;  // rotated channel pairs of a row (d / 2)

// cos and sin of position * f.  A float product is off by up to 2^-24 of
// itself, which at position 2^17 is 2^-7 radian; so the product and the
// removal of whole turns are done in fp64 (the product of a 32-bit position
// and a 24-bit significand is exact to 2^-53), and only the fraction of a
// turn, at most one half, goes to fp32: its rounding moves the angle by at
// most pi * 2^-24.
__device__ __forceinline__ float2 turn(int64_t pos, float f) {
  const double t = (double)pos * (double)f * 0.15915494309189535;  // 1 / (2 pi)
  const float r = (float)(t - rint(t));
  float s, c;
  sincospif(2.0f * r, &s, &c);
  return make_float2(c, s);
}

// Sequence that owns packed row n: the largest b with begin[b] <= n, found by
// the warp 32 probes at a time; -1 when begin[b + 1] <= n or none starts
// at or below n.
__device__ __forceinline__ int owner(const BatchView& bt, int64_t n) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = bt.B;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int p = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, p < hi && bt.begin[p] <= n);
    if (m == 0) return -1;
    const int top = 31 - __clz(m);
    lo += top * step;
    hi = min(hi, lo + step);
  }
  return bt.begin[lo] <= n && n < bt.begin[lo + 1] ? lo : -1;
}

enum Sink { kDense = 0, kPoolRaw = 1, kPoolE4m3 = 2 };

template <typename T, int E>
struct Pack;  // E elements of T as one 16-byte word
template <>
struct Pack<float, 4> {
  __device__ static void unpack(uint4 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  __device__ static void unpack(uint4 a, float (&x)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// Exponent byte of a row whose largest |x| has the bits `top`: the least e
// with |x| <= 448 * 2^e (448 = 1.75 * 2^8), clamped to [-120, 119], as e + 127;
// 255 when |x| is infinite or NaN.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < -120 ? -120 : e > 119 ? 119 : e;
  return e + 127;
}

// One warp per (token, share of its heads); a row of d channels is held by
// LPR lanes, 16 bytes each, so a pass of the warp covers 32 / LPR rows (heads)
// of the token.  The token's angles are computed once by the warp and stay in
// registers over its rows.  Traffic: every row is read once and written once
// (memory bound; the arithmetic of a pass, about 100 instructions for 2 rows
// of 128 bf16, stays below the time its 1 KB takes).
template <typename T, int D, int SINK>
__global__ void __launch_bounds__(128) append_rows_kernel(AppendArgs a) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int LPR = D / E, RPW = 32 / LPR;
  __shared__ float2 tab[4][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR, e0 = li * E;

  if (SINK != kDense && a.status && blockIdx.x == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < a.batch.B; b += blockDim.x) bad |= !seq_view(a.batch, a.pool.shift, b).ok;
    if (bad) set_status(a.status, LOD_ST_BAD_SEQLEN);
  }
  const int64_t job = (int64_t)blockIdx.x * 4 + warp;
  const int64_t n = job / a.split;
  const int part = (int)(job % a.split);
  if (n >= a.N) return;

  // where the token goes
  int64_t b, t, pos, blk = 0;
  bool store = true;
  if constexpr (SINK == kDense) {
    b = n / a.n_new;
    t = n % a.n_new;
    const int64_t len = a.seq_lens[b];
    if (len < a.n_new || len > a.Tmax) return;
    pos = len - a.n_new + t;
  } else {
    const int ob = owner(a.batch, n);
    if (ob < 0) return;
    const SeqView s = seq_view(a.batch, a.pool.shift, ob);
    if (!s.ok) return;
    b = 0;
    t = n;
    pos = s.len - s.n + (n - s.r0);
    blk = a.batch.table[(int64_t)ob * a.batch.max_blocks + (pos >> a.pool.shift)];
    if (blk < 0 || blk >= a.pool.blocks) {
      if (lane == 0) set_status(a.status, LOD_ST_BAD_PAGE);
      store = false;
    }
  }

  // this lane's angles and weights
  float c[E], s[E], wq[E], wk[E];
  const int half = a.use_rope ? a.rope.rot >> 1 : 0, rot = 2 * half;
  const bool inter = a.rope.interleaved != 0;
  for (int i = lane; i < half; i += 32) tab[warp][i] = turn(pos, a.rope.freq[i]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = e0 + i;
    c[i] = 1.f;
    s[i] = 0.f;
    wq[i] = wk[i] = 1.f;
    if (e < rot) {
      const bool second = inter ? (e & 1) : e >= half;
      const float2 cs = tab[warp][inter ? e >> 1 : second ? e - half : e];
      c[i] = cs.x;
      s[i] = second ? cs.y : -cs.y;
    }
  }
  const bool nq = a.use_rope && a.rope.wq, nk = a.use_rope && a.rope.wk;
  if (nq) Pack<T, E>::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.rope.wq) + e0), wq);
  if (nk) Pack<T, E>::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.rope.wk) + e0), wk);
  const bool by_shuffle = !inter && half % E == 0;  // the partner channels sit in one other lane
  const int other = sub * LPR + (e0 < half ? li + half / E : li - half / E);
  const int src = e0 < rot ? other & 31 : lane;

  const int rows = a.Hq + 2 * a.Hkv;
  const int passes = (rows + RPW - 1) / RPW;
  const int p0 = (int)((int64_t)passes * part / a.split), p1 = (int)((int64_t)passes * (part + 1) / a.split);
  auto row_ptr = [&](int r) -> const T* {
    if (r < a.Hq) return static_cast<const T*>(a.q) + b * a.qb + t * a.qt + (int64_t)r * a.qh;
    const bool is_k = r < a.Hq + a.Hkv;
    const T* base = static_cast<const T*>(is_k ? a.k : a.v);
    return base + b * a.kb + t * a.kt + (int64_t)(r - a.Hq - (is_k ? 0 : a.Hkv)) * a.kh;
  };
  auto fetch = [&](int p) -> uint4 {
    const int r = p * RPW + sub;
    return p < p1 && r < rows ? *reinterpret_cast<const uint4*>(row_ptr(r) + e0) : make_uint4(0, 0, 0, 0);
  };
  uint4 raw = fetch(p0);
  for (int p = p0; p < p1; ++p) {
    const uint4 cur = raw;
    raw = fetch(p + 1);
    const int r = p * RPW + sub;
    const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv, live = r < rows;
    float x[E];
    Pack<T, E>::unpack(cur, x);
    if (a.use_rope && __any_sync(0xffffffffu, live && !is_v)) {
      const bool normed = is_q ? nq : nk && !is_v;
      float rstd = 1.f;
      if (nq || nk) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rstd = rsqrtf(ss * (1.f / D) + a.rope.eps);
      }
      float y[E], z[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = normed ? x[i] * rstd * (is_q ? wq[i] : wk[i]) : x[i];
      if (inter) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = y[i ^ 1];
      } else if (by_shuffle) {
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], src);
      } else {
        // a pair's channels at an odd distance: the partners come from the row itself
        const T* xr = row_ptr(live ? r : rows - 1);
        const T* w = static_cast<const T*>(is_q ? a.rope.wq : a.rope.wk);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int e = e0 + i, pe = e < half ? e + half : e - half;
          z[i] = 0.f;
          if (e < rot) z[i] = Elem<T>::to_f(xr[pe]) * (normed ? rstd * Elem<T>::to_f(w[pe]) : 1.f);
        }
        __syncwarp();  // q_out may be q: all partners are read before a row is stored
      }
      if (!is_v) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = e0 + i < rot ? fmaf(z[i], s[i], y[i] * c[i]) : y[i];
      }
    }
    uint32_t top = 0;
    if constexpr (SINK == kPoolE4m3) {
#pragma unroll
      for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (!live) continue;
    if (is_q) {
      *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + b * a.ob + t * a.ot + (int64_t)r * a.oh + e0) =
          Pack<T, E>::pack(x);
      continue;
    }
    const int h = r - a.Hq - (is_v ? a.Hkv : 0);
    if constexpr (SINK == kDense) {
      T* dst = static_cast<T*>(is_v ? a.V : a.K) + b * a.sb + h * a.sh + pos * a.st + e0;
      *reinterpret_cast<uint4*>(dst) = Pack<T, E>::pack(x);
    } else if (store) {
      const int64_t row = ((blk * a.Hkv + h) << a.pool.shift) + (pos & (((int64_t)1 << a.pool.shift) - 1));
      if constexpr (SINK == kPoolRaw) {
        *reinterpret_cast<uint4*>(static_cast<T*>(is_v ? a.pool.V : a.pool.K) + row * D + e0) = Pack<T, E>::pack(x);
      } else {
        const int E8 = row_exponent(top);
        // 2^-e, an fp32 normal over the whole of [-120, 119]: the product is exact (bf16 or fp32 x; tiny
        // x below fp32's normals keep their bits, as the product is larger)
        const float f = __uint_as_float((uint32_t)(254 - (E8 == 255 ? 127 : E8)) << 23);
        uint32_t w[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * f, x[4 * i + 1] * f), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi =
              __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * f, x[4 * i + 3] * f), __NV_SATFINITE, __NV_E4M3);
          w[i] = E8 == 255 ? 0x7f7f7f7fu : lo | (hi << 16);
        }
        uint8_t* dst = static_cast<uint8_t*>(is_v ? a.pool.V : a.pool.K) + row * D + e0;
        if constexpr (E == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = w[0];
        if (li == 0) (is_v ? a.pool.Ve : a.pool.Ke)[row] = (uint8_t)E8;
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_append_t(const AppendArgs& a, int sink, int64_t grid, cudaStream_t st) {
  if (sink == kDense) append_rows_kernel<T, D, kDense><<<(unsigned)grid, 128, 0, st>>>(a);
  else if (sink == kPoolRaw) append_rows_kernel<T, D, kPoolRaw><<<(unsigned)grid, 128, 0, st>>>(a);
  else append_rows_kernel<T, D, kPoolE4m3><<<(unsigned)grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- read-back

// One CTA per (64 consecutive tokens, KV head, sequence): rows of 16-byte
// output pieces, keys and values.  Memory bound: a stored row is read once and
// a dense row written once.
constexpr int kReadTokens = 64;

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(128) pool_read_kernel(ReadArgs a) {
  constexpr int E = 16 / (int)sizeof(T);  // channels of a piece
  constexpr int PPR = D / E;              // pieces of a row
  constexpr int RPP = 128 / PPR;          // rows of a pass of the CTA
  const int b = blockIdx.z, h = blockIdx.y;
  int64_t len = a.batch.seq_lens[b];
  const bool ok = len >= 0 && len <= ((int64_t)a.batch.max_blocks << a.pool.shift);
  if (!ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) set_status(a.status, LOD_ST_BAD_SEQLEN);
    return;
  }
  const int64_t t0 = a.t_begin + (int64_t)blockIdx.x * kReadTokens;
  int64_t t1 = t0 + kReadTokens;
  if (t1 > a.t_end) t1 = a.t_end;
  if (t1 > len) t1 = len;
  if (t0 >= t1) return;
  const int c = threadIdx.x % PPR, r = threadIdx.x / PPR;
  const int64_t mask = ((int64_t)1 << a.pool.shift) - 1;
  const int32_t* table = a.batch.table + (int64_t)b * a.batch.max_blocks;
#pragma unroll 4
  for (int64_t t = t0 + r; t < t1; t += RPP) {
    const int64_t blk = table[t >> a.pool.shift];
    if (blk < 0 || blk >= a.pool.blocks) {
      if (c == 0) set_status(a.status, LOD_ST_BAD_PAGE);
      continue;
    }
    const int64_t row = ((blk * a.pool.Hkv + h) << a.pool.shift) + (t & mask);
    const int64_t dst = b * a.sb + h * a.sh + t * a.st + c * E;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const void* base = kv ? a.pool.V : a.pool.K;
      T* out = static_cast<T*>(kv ? a.V : a.K) + dst;
      if constexpr (!Q8) {
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + row * D + c * E);
      } else {
        const uint8_t* src = static_cast<const uint8_t*>(base) + row * D + c * E;
        uint32_t w[E / 4];
        if constexpr (E == 8) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          w[0] = x.x;
          w[1] = x.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(src);
        }
        const int E8 = (kv ? a.pool.Ve : a.pool.Ke)[row];
        const float f = E8 == 255 ? NAN : E8 == 0 ? __uint_as_float(0x400000u) : __uint_as_float((uint32_t)E8 << 23);
        float x[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
          const float2 v = __half22float2(__half2(hr));
          x[2 * i] = v.x * f;
          x[2 * i + 1] = v.y * f;
        }
        *reinterpret_cast<uint4*>(out) = Pack<T, E>::pack(x);
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_read_t(const ReadArgs& a, int bits, cudaStream_t st) {
  const int64_t tiles = (a.t_end - a.t_begin + kReadTokens - 1) / kReadTokens;
  const dim3 grid((unsigned)tiles, (unsigned)a.pool.Hkv, (unsigned)a.batch.B);
  if (bits == 8) pool_read_kernel<T, D, true><<<grid, 128, 0, st>>>(a);
  else pool_read_kernel<T, D, false><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rows(const AppendArgs& args, int dtype, int d, bool pool, int bits, cudaStream_t stream) {
  AppendArgs a = args;
  // Warps per token: one, unless the call has few tokens; then a token's heads
  // are shared out until the GPU has about 16 warps per SM or every warp has
  // one pass.
  const int elem = dtype == LOD_DTYPE_F32 ? 4 : 2;
  const int rpw = 32 / (d * elem / 16);
  const int passes = (a.Hq + 2 * a.Hkv + rpw - 1) / rpw;
  int64_t split = (int64_t)148 * 16 / a.N;
  if (split > passes) split = passes;
  if (split < 1) split = 1;
  a.split = (int)split;
  const int64_t grid = (a.N * split + 3) / 4;
  const int sink = !pool ? kDense : bits == 8 ? kPoolE4m3 : kPoolRaw;
  if (dtype == LOD_DTYPE_F32)
    return d == 64 ? launch_append_t<float, 64>(a, sink, grid, stream) : launch_append_t<float, 128>(a, sink, grid, stream);
  return d == 64 ? launch_append_t<__nv_bfloat16, 64>(a, sink, grid, stream)
                 : launch_append_t<__nv_bfloat16, 128>(a, sink, grid, stream);
}

cudaError_t launch_pool_read(const ReadArgs& a, int dtype, int bits, int d, cudaStream_t stream) {
  if (dtype == LOD_DTYPE_F32)
    return d == 64 ? launch_read_t<float, 64>(a, bits, stream) : launch_read_t<float, 128>(a, bits, stream);
  return d == 64 ? launch_read_t<__nv_bfloat16, 64>(a, bits, stream) : launch_read_t<__nv_bfloat16, 128>(a, bits, stream);
}

}  // namespace lod
