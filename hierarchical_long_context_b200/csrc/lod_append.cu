// lod_append.cu -- new tokens' projections into a cache (per-head norm, position
// rotation, 8-bit quantisation in the pass that stores them) and the block
// pool's read-back into a dense cache.
#include <cuda_fp8.h>

#include "lod_host.cuh"
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

// No entry of new_begin before begin[b] lies above it (by a warp).
__device__ __forceinline__ bool rises(const BatchView& bt, int b) {
  const int64_t r0 = bt.begin[b];
  bool above = false;
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < b; i += 32) above |= bt.begin[i] > r0;
  return !__any_sync(0xffffffffu, above);
}

// Sequence that owns packed row n, -1: none.  It begins at or below n, at or
// above every earlier entry, and is the first that ends behind n.  Where
// new_begin does not fall (`falls`, of the whole batch) that is the largest b
// with begin[b] <= n, which the warp finds 32 probes at a time; where it does,
// all are looked at.
__device__ __forceinline__ int owner(const BatchView& bt, int64_t n, bool falls) {
  const int lane = threadIdx.x & 31;
  if (falls) {
#pragma unroll 1
    for (int b0 = 0; b0 < bt.B; b0 += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, b0 + lane < bt.B && bt.begin[b0 + lane + 1] > n);
      if (m == 0) continue;
      const int b = b0 + __ffs(m) - 1;
      return bt.begin[b] <= n && rises(bt, b) ? b : -1;
    }
    return -1;
  }
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

// Where a token of the call comes from and goes to; ok = false: nowhere.
struct Place {
  int64_t b, t, pos, blk;  // sequence and token of its strides, position, block
  bool ok, store;          // store = false: a bad block, only q_out is written
};
template <int SINK>
__device__ __forceinline__ Place locate(const AppendArgs& a, int64_t n, bool falls) {
  Place p = {0, n, 0, 0, false, true};
  if (n >= a.N) return p;
  if constexpr (SINK == kDense) {
    p.b = n / a.n_new;
    p.t = n % a.n_new;
    const int64_t len = a.seq_lens[p.b];
    p.ok = len >= a.n_new && len <= a.Tmax;
    p.pos = len - a.n_new + p.t;
  } else {
    const int ob = owner(a.batch, n, falls);
    if (ob < 0) return p;
    const SeqView s = seq_view(a.batch, a.pool.shift, ob);
    if (!s.ok) return p;
    p.ok = true;
    p.pos = s.len - s.n + (n - s.r0);
    p.blk = a.batch.table[(int64_t)ob * a.batch.max_blocks + (p.pos >> a.pool.shift)];
    p.store = p.blk >= 0 && p.blk < a.pool.blocks;
  }
  return p;
}

// One warp per (token, share of its heads); a row of d channels is held by
// LPR lanes, 16 bytes each, so a pass of the warp covers 32 / LPR rows (heads)
// of the token, and the next kBatch passes' rows are loaded while those are
// worked on.  The rows go
// by kind (queries, keys, values).  For a kind, a channel's cosine is
// multiplied by its norm weight and its sine by its partner's once, so that a
// row takes out = rstd * (x * cw + partner * sw): the partners cross lanes as
// the stored 16-byte words, not as floats.  Every row is read once and written
// once.  32768 tokens of 32 + 16 heads, 128 bf16 channels (805 MB in and out):
// 213 us, 58 % of the measured copy rate; without norm and rotation 178 us,
// so the issue of about 75 instructions a pass and the latency at a token's
// start bound it, not the bytes (the six CTAs an SM cost up to 80 bytes of
// spills a thread in the bf16 forms).  Measured and dropped: batches of 4 (220), 8
// CTAs an SM (223), tokens in a loop over warps that keep their weights (230),
// one flat loop over the passes of all kinds (258).
template <typename T, int D, int SINK>
__device__ __forceinline__ void append_token(const AppendArgs& a, float2* tab, int64_t job, const Place& p) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int LPR = D / E, RPW = 32 / LPR;
  constexpr int kBatch = 2;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR, e0 = li * E;
  const int part = (int)(job % a.split);
  if (SINK != kDense && !p.store && lane == 0) set_status(a.status, LOD_ST_BAD_PAGE);
  const int64_t b = p.b, t = p.t, pos = p.pos, blk = p.blk;
  const bool store = p.store;
  const int64_t in_block = pos & (((int64_t)1 << a.pool.shift) - 1);

  // the passes of queries, keys and values, and this warp's share of them
  const int pq = (a.Hq + RPW - 1) / RPW, pk = (a.Hkv + RPW - 1) / RPW, passes = pq + 2 * pk;
  const int p0 = (int)((int64_t)passes * part / a.split), p1 = (int)((int64_t)passes * (part + 1) / a.split);

  const int half = a.use_rope ? a.rope.rot >> 1 : 0, rot = 2 * half;
  const bool inter = a.rope.interleaved != 0;
  if (p0 < pq + pk) {
    for (int i = lane; i < half; i += 32) tab[i] = turn(pos, a.rope.freq[i]);
    __syncwarp();
  }
  const bool by_shuffle = !inter && half % E == 0;  // the partner channels sit in one other lane
  const int src = e0 >= rot ? lane : sub * LPR + (e0 < half ? li + half / E : li - half / E);

#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {  // queries, keys, values
    const int rows = kind == 0 ? a.Hq : a.Hkv, first = kind == 0 ? 0 : kind == 1 ? pq : pq + pk;
    const int count = kind == 0 ? pq : pk;
    const int lo = p0 > first ? p0 - first : 0, hi = p1 < first + count ? p1 - first : count;
    if (lo >= hi) continue;
    const T* in = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
    in += kind == 0 ? b * a.qb + t * a.qt : b * a.kb + t * a.kt;
    const int64_t row_stride = kind == 0 ? a.qh : a.kh;
    const T* w = !a.use_rope || kind == 2 ? nullptr : static_cast<const T*>(kind == 0 ? a.rope.wq : a.rope.wk);
    const bool turned = a.use_rope && kind < 2;

    float cw[E], sw[E];  // cosine times own weight, sine (signed) times the partner's
    if (turned) {
      float own[E];
#pragma unroll
      for (int i = 0; i < E; ++i) own[i] = 1.f;
      if (w) Pack<T, E>::unpack(*reinterpret_cast<const uint4*>(w + e0), own);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = e0 + i;
        cw[i] = own[i];
        sw[i] = 0.f;
        if (e < rot) {
          const bool second = inter ? (e & 1) : e >= half;
          const float2 cs = tab[inter ? e >> 1 : second ? e - half : e];
          const int pe = inter ? e ^ 1 : second ? e - half : e + half;
          cw[i] *= cs.x;
          sw[i] = (second ? cs.y : -cs.y) * (w ? Elem<T>::to_f(w[pe]) : 1.f);
        }
      }
    }
    uint4 ahead[kBatch];  // the next batch's rows: loaded while a batch is worked on
    auto load = [&](int pb) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = (pb + k) * RPW + sub;
        ahead[k] = pb + k < hi && r < rows ? *reinterpret_cast<const uint4*>(in + r * row_stride + e0)
                                           : make_uint4(0, 0, 0, 0);
      }
    };
    load(lo);
    for (int pb = lo; pb < hi; pb += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) raw[k] = ahead[k];
      load(pb + kBatch);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (pb + k >= hi) break;
        const int r = (pb + k) * RPW + sub;
        const bool live = r < rows;
        float x[E];
        Pack<T, E>::unpack(raw[k], x);
        if (turned) {
          float rstd = 1.f;
          if (w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rstd = rsqrtf(ss * (1.f / D) + a.rope.eps);
          }
          float z[E];
          if (inter) {
#pragma unroll
            for (int i = 0; i < E; ++i) z[i] = x[i ^ 1];
          } else if (by_shuffle) {
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, raw[k].x, src);
            o.y = __shfl_sync(0xffffffffu, raw[k].y, src);
            o.z = __shfl_sync(0xffffffffu, raw[k].z, src);
            o.w = __shfl_sync(0xffffffffu, raw[k].w, src);
            Pack<T, E>::unpack(o, z);
          } else {
            // a pair's channels at a distance no 16-byte word divides: the
            // partners come from the row itself
            const T* xr = in + (live ? r : rows - 1) * row_stride;
#pragma unroll
            for (int i = 0; i < E; ++i) {
              const int e = e0 + i;
              z[i] = e < rot ? Elem<T>::to_f(xr[e < half ? e + half : e - half]) : 0.f;
            }
            __syncwarp();  // q_out may be q: all partners are read before a row is stored
          }
#pragma unroll
          for (int i = 0; i < E; ++i) {
            // (a channel that is not turned takes no partner: 0 times an infinity is NaN)
            const float y = x[i] * cw[i];
            x[i] = (e0 + i < rot ? fmaf(z[i], sw[i], y) : y) * rstd;
          }
        }
        if (kind == 0) {
          if (live)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + b * a.ob + t * a.ot + r * a.oh + e0) =
                Pack<T, E>::pack(x);
          continue;
        }
        if constexpr (SINK == kDense) {
          if (live)
            *reinterpret_cast<uint4*>(static_cast<T*>(kind == 2 ? a.V : a.K) + b * a.sb + r * a.sh + pos * a.st + e0) =
                kind == 2 ? raw[k] : Pack<T, E>::pack(x);
        } else {
          const int64_t row = ((blk * a.Hkv + r) << a.pool.shift) + in_block;
          if constexpr (SINK == kPoolRaw) {
            if (live && store)
              *reinterpret_cast<uint4*>(static_cast<T*>(kind == 2 ? a.pool.V : a.pool.K) + row * D + e0) =
                  kind == 2 ? raw[k] : Pack<T, E>::pack(x);
          } else {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int E8 = row_exponent(top);
            // 2^-e, an fp32 normal over the whole of [-120, 119]: the product is exact (bf16 or fp32 x; tiny
            // x below fp32's normals keep their bits, as the product is larger)
            const float f = __uint_as_float((uint32_t)(254 - (E8 == 255 ? 127 : E8)) << 23);
            uint32_t c[E / 4];
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
              const uint32_t l2 =
                  __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * f, x[4 * i + 1] * f), __NV_SATFINITE, __NV_E4M3);
              const uint32_t h2 =
                  __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * f, x[4 * i + 3] * f), __NV_SATFINITE, __NV_E4M3);
              c[i] = E8 == 255 ? 0x7f7f7f7fu : l2 | (h2 << 16);
            }
            if (live && store) {
              uint8_t* dst = static_cast<uint8_t*>(kind == 2 ? a.pool.V : a.pool.K) + row * D + e0;
              if constexpr (E == 8)
                *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
              else
                *reinterpret_cast<uint32_t*>(dst) = c[0];
              if (li == 0) (kind == 2 ? a.pool.Ve : a.pool.Ke)[row] = (uint8_t)E8;
            }
          }
        }
      }
    }
  }
}

// A CTA of a pool's append looks once whether new_begin falls.  Of few
// sequences every CTA does, for its four warps' one token each, and while it
// looks for the tokens' sequences as if it did not fall.  Of many (kMany) the
// grid fits the GPU and the warps take their tokens in turn, as the look costs
// more than a token (65535 sequences of one token: 182 us without it, 220
// so, 1140 with a look of every warp; 2048: 19.1, 21.1).
constexpr int kManySeqs = 1024;
template <typename T, int D, int SINK, bool kMany>
__global__ void __launch_bounds__(128, 6) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 tab[4][kMaxPairs];
  const int warp = threadIdx.x >> 5;
  int64_t job = (int64_t)blockIdx.x * 4 + warp;
  bool falls = false;
  const int64_t* begin = a.batch.begin;
  const int B = a.batch.B;
  if constexpr (kMany) {
#pragma unroll 8
    for (int i = threadIdx.x + 1; i < B; i += 128) falls |= begin[i] < begin[i - 1];
    falls = __syncthreads_or(falls);
    for (; job < a.N * a.split; job += (int64_t)gridDim.x * 4) {
      const Place p = locate<SINK>(a, job / a.split, falls);
      if (p.ok) append_token<T, D, SINK>(a, tab[warp], job, p);
      __syncwarp();  // (tab)
    }
  } else {
    // (the first entries are on their way while the tokens are looked for; up
    // to 33 a warp looks at by itself, without the CTA's barrier)
    int64_t x[4], y[4];
    const int i0 = SINK != kDense && B <= 33 ? threadIdx.x & 31 : threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 128 * k;
      x[k] = y[k] = 0;
      if (SINK != kDense && i + 1 < B) x[k] = begin[i], y[k] = begin[i + 1];
    }
    Place p = locate<SINK>(a, job / a.split, false);
    if constexpr (SINK != kDense) {
#pragma unroll
      for (int k = 0; k < 4; ++k) falls |= y[k] < x[k];
#pragma unroll 4
      for (int i = i0 + 513; i < B; i += 128) falls |= begin[i] < begin[i - 1];
      falls = B <= 33 ? __any_sync(0xffffffffu, falls) != 0 : __syncthreads_or(falls) != 0;
      if (falls) p = locate<SINK>(a, job / a.split, true);
    }
    if (p.ok) append_token<T, D, SINK>(a, tab[warp], job, p);
  }
  if (SINK != kDense && a.status && blockIdx.x == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < B; b += 128) bad |= !seq_view(a.batch, a.pool.shift, b).ok;
    if (bad) set_status(a.status, LOD_ST_BAD_SEQLEN);
  }
}

template <typename T, int D, int SINK>
cudaError_t launch_append_sink(const AppendArgs& a, int64_t grid, cudaStream_t st) {
  const int64_t fit = (int64_t)host::num_sms() * 6;
  if (SINK != kDense && a.batch.B > kManySeqs && grid > fit)
    append_rows_kernel<T, D, SINK == kDense ? kPoolRaw : SINK, true><<<(unsigned)fit, 128, 0, st>>>(a);
  else
    append_rows_kernel<T, D, SINK, false><<<(unsigned)grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_append_t(const AppendArgs& a, int sink, int64_t grid, cudaStream_t st) {
  if (sink == kDense) return launch_append_sink<T, D, kDense>(a, grid, st);
  return sink == kPoolRaw ? launch_append_sink<T, D, kPoolRaw>(a, grid, st) : launch_append_sink<T, D, kPoolE4m3>(a, grid, st);
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
  constexpr int PASSES = kReadTokens / RPP;  // rows of a thread
  constexpr int BATCH = PASSES < 4 ? PASSES : 4;
#pragma unroll 1
  for (int p0 = 0; p0 < PASSES; p0 += BATCH) {
    // the rows of a batch first, then all their loads, then the stores
    int64_t row[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int64_t t = t0 + r + (int64_t)(p0 + k) * RPP;
      row[k] = -1;
      if (t < t1) {
        const int64_t blk = table[t >> a.pool.shift];
        if (blk >= 0 && blk < a.pool.blocks)
          row[k] = ((blk * a.pool.Hkv + h) << a.pool.shift) + (t & mask);
        else if (c == 0)
          set_status(a.status, LOD_ST_BAD_PAGE);
      }
    }
    uint4 x[BATCH][2];
    int E8[BATCH][2];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (row[k] < 0) continue;
        const void* base = kv ? a.pool.V : a.pool.K;
        if constexpr (!Q8) {
          x[k][kv] = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + row[k] * D + c * E);
        } else {
          const uint8_t* src = static_cast<const uint8_t*>(base) + row[k] * D + c * E;
          E8[k][kv] = (kv ? a.pool.Ve : a.pool.Ke)[row[k]];
          if constexpr (E == 8) {
            const uint2 w = *reinterpret_cast<const uint2*>(src);
            x[k][kv].x = w.x;
            x[k][kv].y = w.y;
          } else {
            x[k][kv].x = *reinterpret_cast<const uint32_t*>(src);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (row[k] < 0) continue;
      const int64_t t = t0 + r + (int64_t)(p0 + k) * RPP;
      const int64_t dst = b * a.sb + h * a.sh + t * a.st + c * E;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(kv ? a.V : a.K) + dst);
        if constexpr (!Q8) {
          *out = x[k][kv];
        } else {
          const int e = E8[k][kv];
          const float f = e == 255 ? NAN : e == 0 ? __uint_as_float(0x400000u) : __uint_as_float((uint32_t)e << 23);
          const uint32_t w[2] = {x[k][kv].x, x[k][kv].y};
          float y[E];
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const __half2_raw hr =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
            const float2 v = __half22float2(__half2(hr));
            y[2 * i] = v.x * f;
            y[2 * i + 1] = v.y * f;
          }
          *out = Pack<T, E>::pack(y);
        }
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
  const int passes = (a.Hq + rpw - 1) / rpw + 2 * ((a.Hkv + rpw - 1) / rpw);
  int64_t split = (int64_t)host::num_sms() * 16 / a.N;
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
