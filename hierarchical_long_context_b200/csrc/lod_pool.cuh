// lod_pool.cuh -- argument blocks, launchers and shared device code of the
// block pool (append with norm and rotation, read-back, exact attention).
#pragma once

#include <cuda.h>

#include "lod_internal.cuh"

namespace lod {

// The device side of a lod_batch.
struct BatchView {
  const int32_t* table;     // [B][max_blocks]
  const int64_t* seq_lens;  // [B]
  const int64_t* begin;     // [B + 1] (null for lod_pool_read)
  int64_t N, max_new;
  int B, max_blocks;
};

// The device side of a lod_pool.
struct PoolView {
  void* K;
  void* V;
  uint8_t* Ke;
  uint8_t* Ve;
  int64_t blocks;
  int Hkv;
  int shift;  // log2(block)
};

struct RopeView {
  const void* wq;
  const void* wk;
  const float* freq;
  float eps;
  int rot;
  int interleaved;
};

// Rows of new tokens on their way into a cache.
struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t qb, qh, qt, kb, kh, kt, ob, oh, ot;  // strides in elements (sequence, head, token)
  int Hq, Hkv;          // Hq = 0: no queries
  int use_rope;
  RopeView rope;
  int64_t N;            // tokens of the call
  int split;            // warps that share one token's heads
  // dense cache
  void* K;
  void* V;
  int64_t sb, sh, st, Tmax, n_new;
  const int64_t* seq_lens;
  // pool
  PoolView pool;
  BatchView batch;
  uint32_t* status;
};

struct ReadArgs {
  PoolView pool;
  BatchView batch;
  void* K;
  void* V;
  int64_t sb, sh, st, t_begin, t_end;
  uint32_t* status;
};

// Exact attention over the pool.  A work unit is (sequence, KV head, tile of
// TM query rows); row r of a sequence and KV head is query head r % G of its
// new token r / G.  A unit's keys are cut into tiles of KT; the tiles of all
// units, in the order sequence, head, row tile, key tile, are one list, and
// CTA c takes the entries [c * share, (c + 1) * share) of it.  Each unit opens
// with kUnitCost entries that hold no tile: what a unit costs beside its tiles
// (queries, first maxima, results).  Without them a CTA that gets a batch's
// short sequences was the last to finish (150 us for 79 tiles, against 100).
constexpr int kUnitCost = 3;
struct PoolAttendArgs {
  const void* q;
  void* out;
  float* lse;
  int64_t qt, qh, ot, oh;  // strides in elements (token, head)
  PoolView pool;
  BatchView batch;
  int Hq, G;
  int64_t window;          // 0: none
  float scale_log2;        // softmax scale * log2 e
  // workspace
  uint32_t* status;
  int64_t* Wb;             // [B + 1] key tiles before each sequence (all heads)
  int32_t* RT;             // [B + 1] row tiles before each sequence (one head)
  int32_t* pre;            // [RT[B]] key tiles of the sequence (one head) before each row tile
  float* part;             // [parts][2][TM][d] partial sums
  float2* ml;              // [parts][2][TM] their (max, sum), log2 units
  struct MergeRec* rec;    // [parts] the unit that opens in a part and goes on behind it
  int ctas;
  int planned;             // 1: Wb, RT, pre were written by the plan kernel
  // The kernel of many rows takes the list in rounds: a CTA's parts are c, c +
  // ctas, ... of ctas * rounds.  The CTAs of a round then read about
  // kRoundBytes of the cache between them, which stays in L2 while the
  // row tiles of a head sweep over it at offsets of their own (a 2048-token
  // chunk over 128K read 15.8 GB from DRAM in one round, for 0.54 GB of cache;
  // rounds of 64 MB take 4.31 ms, of 96 MB 4.55, of 40 MB 4.31).
  int max_rounds;
  int32_t* rounds;         // (null: one round)
  int row_bytes;           // stored bytes of a key and its value
};
constexpr int64_t kRoundBytes = (int64_t)64 << 20;
constexpr int kMaxRounds = 8;

// Sequence b of a batch, checked by itself: [r0, r1) = its packed rows, n = new
// tokens (0 when the sequence is refused), len = tokens.  A sequence that
// begins below an earlier entry of new_begin is refused too, which only those
// who look at the whole batch can tell (the work list, the append's owner).
// Those left have r0 at or above every earlier sequence's r1, so they share no
// row, and their row tiles number at most N * G / TM + B.
struct SeqView {
  int64_t r0, r1, len;
  int n;
  bool ok;
};
__device__ __forceinline__ SeqView seq_view(const BatchView& bt, int shift, int b) {
  SeqView s;
  const int64_t r0 = bt.begin[b], r1 = bt.begin[b + 1];
  s.len = bt.seq_lens[b];
  s.r0 = r0;
  s.r1 = r1;
  s.ok = r0 >= 0 && r1 >= r0 && r1 <= bt.N && r1 - r0 <= bt.max_new && s.len >= r1 - r0 &&
         s.len <= ((int64_t)bt.max_blocks << shift);
  s.n = s.ok ? (int)(r1 - r0) : 0;
  return s;
}

// The same of a sequence that the work list holds, and so is known to be good:
// every role of a CTA walks the list, and the checks in each of them cost
// instruction cache.
__device__ __forceinline__ SeqView seq_taken(const BatchView& bt, int b) {
  SeqView s;
  s.r0 = bt.begin[b];
  s.r1 = bt.begin[b + 1];
  s.len = bt.seq_lens[b];
  s.n = (int)(s.r1 - s.r0);
  s.ok = true;
  return s;
}

// Key tiles [lo, hi) that row tile i (rows [i * TM, ...)) of a sequence reads.
template <int TM, int KT>
__device__ __forceinline__ void row_tile_keys(const SeqView& s, int G, int64_t window, int64_t i, int& lo, int& hi) {
  const int64_t rows = (int64_t)s.n * G;
  int64_t r1 = (i + 1) * TM;
  if (r1 > rows) r1 = rows;
  const int64_t t0 = s.len - s.n + i * TM / G, t1 = s.len - s.n + (r1 - 1) / G;
  int64_t first = window > 0 ? t0 - window + 1 : 0;
  if (first < 0) first = 0;
  lo = (int)(first / KT);
  hi = (int)(t1 / KT) + 1;
}

// Unit that holds an entry of the work list, and the entry's key tile.
struct Unit {
  int b, h;
  int64_t i;        // row tile
  int64_t begin;    // list position of the unit
  int lo, hi;       // its key tiles [lo, hi); entry w is key tile lo + (w - first())
  __device__ __forceinline__ int64_t first() const { return begin + kUnitCost; }
  __device__ __forceinline__ int64_t end() const { return begin + kUnitCost + (hi - lo); }
};

template <int TM, int KT>
__device__ __forceinline__ Unit find_unit(const PoolAttendArgs& a, const int64_t* Wb, int64_t w) {
  Unit u;
  int lo = 0, hi = a.batch.B;  // Wb[lo] <= w < Wb[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (Wb[mid] <= w) lo = mid; else hi = mid;
  }
  u.b = lo;
  const int64_t per_head = (Wb[lo + 1] - Wb[lo]) / a.pool.Hkv;
  u.h = (int)((w - Wb[lo]) / per_head);
  const int64_t head0 = Wb[lo] + u.h * per_head;
  u.i = 0;
  u.begin = head0;
  if (a.planned) {
    const int32_t* pre = a.pre + a.RT[lo];
    int64_t l = 0, r = a.RT[lo + 1] - a.RT[lo];
    while (r - l > 1) {
      const int64_t mid = (l + r) >> 1;
      if (pre[mid] <= w - head0) l = mid; else r = mid;
    }
    u.i = l;
    u.begin = head0 + pre[l];
  }
  const SeqView s = seq_taken(a.batch, u.b);
  row_tile_keys<TM, KT>(s, a.G, a.window, u.i, u.lo, u.hi);
  return u;
}

// What the merge needs of the unit whose first tile lies in a part and whose
// last lies behind it (there is at most one): written by that part's CTA.
// pieces = 0: there is none.
struct __align__(16) MergeRec {
  int pieces, nrow;  // parts it reaches into; its rows
  int g0, head0;     // its first row, its first query head
  int64_t r0;        // packed row of its sequence's first new token
};

// Parts of the list, and the entries of one.
__device__ __forceinline__ int list_parts(const PoolAttendArgs& a) { return a.ctas * (a.rounds ? *a.rounds : 1); }
__device__ __forceinline__ int64_t list_share(const PoolAttendArgs& a, int64_t total) {
  const int parts = list_parts(a);
  return (total + parts - 1) / parts;
}

// A CTA's walk through a part [w, w1) of the list, one piece of a unit at a
// time: key tiles [kt0, kt1) of unit u.  Every role of a CTA takes the same walk.
template <int TM, int KT>
struct Walk {
  const PoolAttendArgs& a;
  const int64_t* Wb;
  int64_t w0, w, w1, uend;
  Unit u;
  SeqView s;
  int64_t pe;       // end of the piece
  int nt, kt0, kt1, nrow;

  __device__ __forceinline__ Walk(const PoolAttendArgs& args, const int64_t* wb, int part) : a(args), Wb(wb) {
    const int64_t total = Wb[a.batch.B], share = list_share(a, total);
    w0 = w = part * share;
    w1 = w0 + share < total ? w0 + share : total;
    if (w < w1) {
      u = find_unit<TM, KT>(a, Wb, w);
      s = seq_taken(a.batch, u.b);
      nt = (s.n * a.G + TM - 1) / TM;
      piece();
      if (kt0 == kt1) next();
    }
  }
  __device__ __forceinline__ bool more() const { return w < w1; }
  __device__ __forceinline__ void piece() {
    uend = u.end();
    pe = uend < w1 ? uend : w1;
    kt0 = u.lo + (w > u.first() ? (int)(w - u.first()) : 0);
    kt1 = u.lo + (pe > u.first() ? (int)(pe - u.first()) : 0);
    const int left = s.n * a.G - (int)u.i * TM;
    nrow = left < TM ? left : TM;
  }
  __device__ __forceinline__ void next() {
    do {
      w = pe;
      if (w >= w1) return;
      u.begin = uend;  // a piece that does not reach its unit's end is the walk's last
      if (u.i + 1 < nt) {
        ++u.i;
      } else {
        u.i = 0;
        if (++u.h == a.pool.Hkv) {
          u.h = 0;
          do ++u.b;
          while (Wb[u.b + 1] == u.begin);  // (no new tokens, or refused)
          s = seq_taken(a.batch, u.b);
          nt = (s.n * a.G + TM - 1) / TM;
        }
      }
      row_tile_keys<TM, KT>(s, a.G, a.window, u.i, u.lo, u.hi);
      piece();
    } while (kt0 == kt1);
  }
  // (after the walk; by one thread)
  __device__ __forceinline__ void record(int part) const {
    MergeRec r = {0, 0, 0, 0, 0};
    if (w0 < w1 && uend > w1 && u.first() >= w0 && u.first() < w1) {
      const int64_t share = list_share(a, Wb[a.batch.B]);
      r = {(int)((uend - 1) / share) - part + 1, nrow, (int)u.i * TM, u.h * a.G, s.r0};
    }
    a.rec[part] = r;
  }
  __device__ __forceinline__ bool whole() const { return w <= u.first() && pe == uend; }
  __device__ __forceinline__ int slot(int part) const { return 2 * part + (u.first() >= w0 ? 1 : 0); }
};

// Sequences a CTA can lay out by itself (one row tile each): the list's
// prefix sums then live in its shared memory and no plan kernel runs.
constexpr int kInlineSeqs = 256;

// Wb of sequences with one row tile each, by the whole CTA (at least one
// warp); ends with a CTA barrier.  The sequences are read side by side, then
// added up by a warp.  While new_begin rises no entry lies above a later one;
// the running maximum is taken only where it falls.
template <int TM, int KT>
__device__ __forceinline__ void plan_inline(const PoolAttendArgs& a, int64_t* Wb) {
  bool falls = false;
  for (int b = threadIdx.x; b < a.batch.B; b += blockDim.x) {
    const SeqView s = seq_view(a.batch, a.pool.shift, b);
    int lo = 0, hi = -kUnitCost;
    if (s.n > 0) row_tile_keys<TM, KT>(s, a.G, a.window, 0, lo, hi);
    Wb[b + 1] = (int64_t)(hi - lo + kUnitCost) * a.pool.Hkv;
    falls |= s.r1 < s.r0;
  }
  falls = __syncthreads_or(falls);
  if (threadIdx.x < 32) {
    int64_t at = 0, top = INT64_MIN;
    if (threadIdx.x == 0) Wb[0] = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch.B; b0 += 32) {
      const int b = b0 + threadIdx.x;
      int64_t n = b < a.batch.B ? Wb[b + 1] : 0;
      if (falls) {
        const int64_t r0 = b < a.batch.B ? a.batch.begin[b] : INT64_MIN;
        int64_t m = r0 > top ? r0 : top;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, m, o);
          if ((int)threadIdx.x >= o && x > m) m = x;
        }
        if (r0 < m) n = 0;
        top = __shfl_sync(0xffffffffu, m, 31);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, n, o);
        if ((int)threadIdx.x >= o) n += x;
      }
      if (b < a.batch.B) Wb[b + 1] = at + n;
      at += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  __syncthreads();
}

// Rows of refused sequences: out = 0, lse = -inf.  A refused sequence may
// name rows of another that is not: of its rows it clears those that no
// earlier sequence reaches.  (The entries of new_begin up to b rise and fall
// from begin[0] to their maximum, so each row between these two is passed by a
// rising pair first: its sequence owns the row, or clears it.)
template <typename T, int D>
__device__ __forceinline__ void clear_rows(const PoolAttendArgs& a, int b) {
  constexpr int N16 = D * (int)sizeof(T) / 16;
  const SeqView s = seq_view(a.batch, a.pool.shift, b);
  if (s.ok && s.n == 0) return;
  if (threadIdx.x == 0) set_status(a.status, LOD_ST_BAD_SEQLEN);
  int64_t top = s.r0;
  for (int i = threadIdx.x & 31; i < b; i += 32)
    if (a.batch.begin[i] > top) top = a.batch.begin[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const int64_t x = __shfl_xor_sync(0xffffffffu, top, o);
    if (x > top) top = x;
  }
  const int64_t end = s.r1 < a.batch.N ? s.r1 : a.batch.N, begin0 = a.batch.begin[0];
#pragma unroll 1
  for (int below = 0; below < 2; ++below) {  // its rows above every earlier entry, and those below the first one
    int64_t r0 = below ? s.r0 : top;
    const int64_t r1 = below && begin0 < end ? begin0 : end;
    if (below && s.r0 >= begin0) break;
    if (r0 < 0) r0 = 0;
    for (int64_t x = threadIdx.x; r0 < r1 && x < (r1 - r0) * a.Hq * N16; x += blockDim.x) {
      const int64_t row = x / N16, t = r0 + row / a.Hq, h = row % a.Hq;
      const int c = (int)(x % N16);
      reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.ot + h * a.oh)[c] = make_uint4(0, 0, 0, 0);
      if (c == 0 && a.lse) a.lse[t * a.Hq + h] = -INFINITY;
    }
  }
}
// (the tensor-core kernels call it: inlined, it lengthens what every warp
// fetches at its start, 1 us of a decode step; the fp32 kernel is 4 % slower
// with a call in it)
template <typename T, int D>
__device__ __noinline__ void clear_rows_call(const PoolAttendArgs& a, int b) {
  clear_rows<T, D>(a, b);
}
// Every CTA of the grid calls this with all its threads; the CTAs share the
// sequences out.
template <typename T, int D, bool kCall>
__device__ __forceinline__ void clear_refused(const PoolAttendArgs& a, const int64_t* Wb) {
  for (int b = blockIdx.x; b < a.batch.B; b += gridDim.x) {
    if (Wb[b + 1] > Wb[b]) continue;
    if (kCall) clear_rows_call<T, D>(a, b);
    else clear_rows<T, D>(a, b);
  }
}

cudaError_t launch_append_rows(const AppendArgs& a, int dtype, int d, bool pool, int bits, cudaStream_t stream);
cudaError_t launch_pool_read(const ReadArgs& a, int dtype, int bits, int d, cudaStream_t stream);

// Shape of an attention call: which kernel, its tiles and its CTAs.
struct PoolShape {
  int kind;  // 0: CUDA cores (fp32); 1: tensor cores, 256 rows a unit; 2: tensor cores, few rows
  int TM, ctas;
  bool inline_plan;
  int max_rounds;
  size_t off_plan, off_ml, off_rec, off_part, total;  // workspace offsets
};
// Stored bytes of a key and its value.
inline int pool_row_bytes(int dtype, int bits, int d) {
  return 2 * (bits == 8 ? d + 1 : d * (dtype == LOD_DTYPE_F32 ? 4 : 2));
}
PoolShape pool_shape(int dtype, int bits, int d, int Hkv, int G, int B, int64_t capacity, int64_t N, int64_t max_new,
                     int sms);
// TMA tensor maps of a bf16 pool's K and V: rows x d, boxes of 64 channels x one block.
struct __align__(64) PoolMaps {
  CUtensorMap K, V;
};
// Tensor cores, many rows: bf16 rows or e4m3 codes.
cudaError_t launch_pool_rows(const PoolAttendArgs& a, const PoolMaps* maps, int bits, int d, cudaStream_t stream);
// Tensor cores, at most TM = 8, 16, 32 or 64 rows per sequence and KV head.
cudaError_t launch_pool_few(const PoolAttendArgs& a, const PoolMaps* maps, int TM, int bits, int d, cudaStream_t stream);

cudaError_t launch_pool_attend(PoolAttendArgs& a, const PoolShape& s, const PoolMaps* maps, int dtype, int bits, int d,
                               cudaStream_t stream);

}  // namespace lod
