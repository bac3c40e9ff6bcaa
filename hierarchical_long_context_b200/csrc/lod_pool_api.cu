// lod_pool_api.cu -- the extern "C" entry points of the projections' append and
// of the block pool (include/lod.h): argument checks, workspace layout, launches.
#include <cmath>
#include <cstring>

#include "lod_host.cuh"
#include "lod_pool.cuh"

namespace {

using namespace lod::host;

int64_t elem_of(int32_t dtype) { return dtype == LOD_DTYPE_F32 ? 4 : 2; }

// `count` strides of rows of elem-byte elements: non-negative multiples of 16 bytes.
int32_t check_strides(const int64_t* s, int count, int64_t elem, const char* name) {
  if (!s) return fail(LOD_EINVAL, "%s is NULL", name);
  for (int i = 0; i < count; ++i)
    if (s[i] < 0 || (s[i] * elem) % 16)
      return fail(LOD_EINVAL, "%s[%d] must be a non-negative multiple of 16 bytes", name, i);
  return LOD_OK;
}

// The rows of an output lie apart: taken by rising stride, each dimension
// steps over all that the smaller ones cover (every slice and permutation of a
// contiguous array does).
int32_t check_apart(const int64_t* s, const int64_t* sizes, int count, int64_t d, const char* name) {
  int64_t covered = d, last = -1;
  int at = -1;
  for (int k = 0; k < count; ++k) {
    int next = -1;
    for (int i = 0; i < count; ++i)
      if ((s[i] > last || (s[i] == last && i > at)) &&
          (next < 0 || s[i] < s[next])) next = i;
    last = s[next], at = next;
    if (sizes[next] <= 1) continue;
    if (last < covered || last > (INT64_MAX - covered) / sizes[next])
      return fail(LOD_EINVAL, "%s gives rows that overlap", name);
    covered += last * (sizes[next] - 1);
  }
  return LOD_OK;
}

int32_t check_rope(const lod_rope* r, int32_t d) {
  if (!(r->eps >= 0.f)) return fail(LOD_EINVAL, "rope eps must be >= 0");
  if (r->rot < 0 || r->rot > d || (r->rot & 1)) return fail(LOD_EINVAL, "rope rot = %d must be even, in [0, d]", r->rot);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(LOD_EINVAL, "rope interleaved must be 0 or 1");
  if (r->rot > 0 && !r->inv_freq) return fail(LOD_EINVAL, "rope inv_freq is NULL with rot = %d", r->rot);
  if (reinterpret_cast<uintptr_t>(r->inv_freq) & 3u) return fail(LOD_EINVAL, "rope inv_freq must be 4-byte aligned");
  if (!aligned16(r->q_norm) || !aligned16(r->k_norm)) return fail(LOD_EINVAL, "rope norm weights must be 16-byte aligned");
  return check_visible_all({{r->q_norm, "q_norm"}, {r->k_norm, "k_norm"}, {r->inv_freq, "inv_freq"}});
}

int32_t shift_of(int32_t block) {
  int s = 0;
  while ((1 << s) < block) ++s;
  return s;
}

int32_t check_pool_format(const lod_pool* p) {
  if (!p) return fail(LOD_EINVAL, "pool is NULL");
  if (p->dtype != LOD_DTYPE_F32 && p->dtype != LOD_DTYPE_BF16)
    return fail(LOD_EUNSUPPORTED, "dtype %d unsupported (0=f32, 1=bf16)", p->dtype);
  if (p->bits != 0 && p->bits != 8) return fail(LOD_EUNSUPPORTED, "pool bits = %d unsupported (0 or 8)", p->bits);
  if (p->d != 64 && p->d != 128) return fail(LOD_EUNSUPPORTED, "d = %d unsupported (64 or 128)", p->d);
  if (p->Hq < 1 || p->Hkv < 1) return fail(LOD_EINVAL, "Hq, Hkv must be >= 1");
  if (p->Hq % p->Hkv) return fail(LOD_EINVAL, "Hq (%d) must be a multiple of Hkv (%d)", p->Hq, p->Hkv);
  if (p->Hq / p->Hkv > 64) return fail(LOD_EUNSUPPORTED, "Hq/Hkv = %d exceeds 64", p->Hq / p->Hkv);
  if (p->Hkv > 65535) return fail(LOD_EUNSUPPORTED, "Hkv = %d exceeds 65535", p->Hkv);
  if (p->block != 16 && p->block != 32 && p->block != 64 && p->block != 128)
    return fail(LOD_EUNSUPPORTED, "block = %d unsupported (16, 32, 64 or 128)", p->block);
  if (p->blocks < 1) return fail(LOD_EINVAL, "a pool needs at least one block");
  if (p->blocks > (((int64_t)1 << 31) - 1) / ((int64_t)p->Hkv * p->block))
    return fail(LOD_EUNSUPPORTED, "blocks * Hkv * block must stay below 2^31");
  return LOD_OK;
}

int32_t check_pool(const lod_pool* p) {
  int32_t rc = check_pool_format(p);
  if (rc) return rc;
  if (!p->K || !p->V) return fail(LOD_EINVAL, "pool K and V must be non-NULL");
  if (!aligned16(p->K) || !aligned16(p->V)) return fail(LOD_EINVAL, "pool K and V must be 16-byte aligned");
  if (p->bits == 8 && (!p->Ke || !p->Ve)) return fail(LOD_EINVAL, "an 8-bit pool needs Ke and Ve");
  if (p->bits == 8 && (!aligned16(p->Ke) || !aligned16(p->Ve)))
    return fail(LOD_EINVAL, "pool Ke and Ve must be 16-byte aligned");
  return check_visible_all({{p->K, "pool K"}, {p->V, "pool V"}, {p->bits == 8 ? p->Ke : nullptr, "pool Ke"},
                            {p->bits == 8 ? p->Ve : nullptr, "pool Ve"}});
}

int32_t check_batch_sizes(const lod_pool* p, const lod_batch* b) {
  if (!b) return fail(LOD_EINVAL, "batch is NULL");
  if (b->B < 1 || b->B > 65535) return fail(LOD_EINVAL, "batch B = %d must be in [1, 65535]", b->B);
  if (b->max_blocks < 1 || (int64_t)b->max_blocks * p->block >= ((int64_t)1 << 31))
    return fail(LOD_EINVAL, "batch max_blocks = %d must be >= 1, with max_blocks * block below 2^31", b->max_blocks);
  return LOD_OK;
}

int32_t check_new_rows(const lod_pool* p, const lod_batch* b) {
  if (b->N < 1 || b->N > ((int64_t)1 << 31) / p->Hq - 1)
    return fail(LOD_EINVAL, "batch N = %lld must be >= 1, with N * Hq below 2^31", (long long)b->N);
  if (b->max_new < 1 || b->max_new > b->N)
    return fail(LOD_EINVAL, "batch max_new = %lld must be in [1, N]", (long long)b->max_new);
  // the attention's list counts a sequence's tiles in 32 bits (8 query rows, 64 keys and more a tile)
  const int64_t row_tiles = b->max_new * (p->Hq / p->Hkv) / 8 + 1, key_tiles = (int64_t)b->max_blocks * p->block / 64 + 8;
  if (row_tiles > (((int64_t)1 << 31) - 1) / key_tiles)
    return fail(LOD_EUNSUPPORTED, "max_new = %lld rows over %lld tokens: too many tiles for one call",
                (long long)b->max_new, (long long)b->max_blocks * p->block);
  return LOD_OK;
}

int32_t check_batch(const lod_pool* p, const lod_batch* b, bool rows) {
  int32_t rc = check_batch_sizes(p, b);
  if (!rc && rows) rc = check_new_rows(p, b);
  if (rc) return rc;
  if (!b->block_table || !b->seq_lens || (rows && !b->new_begin))
    return fail(LOD_EINVAL, "batch block_table, seq_lens and new_begin must be non-NULL");
  if ((reinterpret_cast<uintptr_t>(b->block_table) & 3u) || (reinterpret_cast<uintptr_t>(b->seq_lens) & 7u) ||
      (rows && (reinterpret_cast<uintptr_t>(b->new_begin) & 7u)))
    return fail(LOD_EINVAL, "batch block_table, seq_lens or new_begin is misaligned");
  return check_visible_all({{b->block_table, "block_table"}, {b->seq_lens, "seq_lens"},
                            {rows ? b->new_begin : nullptr, "new_begin"}});
}

lod::PoolView pool_view(const lod_pool* p) {
  return {p->K, p->V, p->Ke, p->Ve, p->blocks, p->Hkv, shift_of(p->block)};
}
lod::BatchView batch_view(const lod_batch* b) {
  return {b->block_table, b->seq_lens, b->new_begin, b->N, b->max_new, b->B, b->max_blocks};
}
lod::RopeView rope_view(const lod_rope* r) {
  return {r->q_norm, r->k_norm, r->inv_freq, r->eps, r->rot, r->interleaved};
}

// q and q_out of an append: both or neither, aligned, with `count` strides.
int32_t check_queries(const void* q, const int64_t* qs, const void* q_out, const int64_t* os, const int64_t* sizes,
                      int count, int64_t elem, int64_t d) {
  if (!q != !q_out) return fail(LOD_EINVAL, "q and q_out go together");
  if (!q) return LOD_OK;
  if (!aligned16(q) || !aligned16(q_out)) return fail(LOD_EINVAL, "q and q_out must be 16-byte aligned");
  int32_t rc = check_strides(qs, count, elem, "q_strides");
  if (!rc) rc = check_strides(os, count, elem, "q_out_strides");
  if (!rc) rc = check_apart(os, sizes, count, d, "q_out_strides");
  if (!rc && q == q_out)
    for (int i = 0; i < count; ++i)
      if (qs[i] != os[i]) return fail(LOD_EINVAL, "q_out may be q itself only with the strides of q");
  return rc ? rc : check_visible_all({{q, "q"}, {q_out, "q_out"}});
}

int32_t check_new_kv(const void* k, const void* v, const int64_t* s, int count, int64_t elem) {
  if (!k || !v) return fail(LOD_EINVAL, "k and v must be non-NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(LOD_EINVAL, "k and v must be 16-byte aligned");
  const int32_t rc = check_strides(s, count, elem, "kv_new_strides");
  return rc ? rc : check_visible_all({{k, "k"}, {v, "v"}});
}

int32_t check_status(const uint32_t* status) {
  if (reinterpret_cast<uintptr_t>(status) & 3u) return fail(LOD_EINVAL, "status must be 4-byte aligned");
  return check_visible(status, "status");
}

lod::PoolShape shape_of(const lod_pool* p, const lod_batch* b) {
  return lod::pool_shape(p->dtype, p->bits, p->d, p->Hkv, p->Hq / p->Hkv, b->B, (int64_t)b->max_blocks * p->block, b->N,
                         b->max_new, num_sms());
}

}  // namespace

extern "C" {

int32_t lod_append_rope(const lod_params* p, const lod_rope* rope, const void* q, const int64_t q_strides[3],
                        const void* k, const void* v, const int64_t kv_new_strides[3], int64_t n_new, void* K,
                        void* V, const int64_t kv_strides[3], const int64_t* seq_lens, void* q_out,
                        const int64_t q_out_strides[3], lod_stream_t stream) {
  int32_t rc = check_params(p);
  if (!rc) rc = check_cache(p, K, V, kv_strides);
  if (rc) return rc;
  if (!rope) return fail(LOD_EINVAL, "rope is NULL");
  if (!seq_lens) return fail(LOD_EINVAL, "seq_lens must be non-NULL");
  if (reinterpret_cast<uintptr_t>(seq_lens) & 7u) return fail(LOD_EINVAL, "seq_lens must be 8-byte aligned");
  if (n_new < 1 || n_new > p->Tmax) return fail(LOD_EINVAL, "n_new = %lld must be in [1, Tmax]", (long long)n_new);
  const int64_t elem = elem_of(p->dtype);
  const int64_t N = p->B * n_new;
  if (N >= ((int64_t)1 << 31)) return fail(LOD_EUNSUPPORTED, "B * n_new must stay below 2^31");
  rc = check_rope(rope, p->d);
  const int64_t rows[3] = {p->B, p->Hq, n_new};
  if (!rc) rc = check_queries(q, q_strides, q_out, q_out_strides, rows, 3, elem, p->d);
  if (!rc) rc = check_new_kv(k, v, kv_new_strides, 3, elem);
  const int64_t cached[3] = {p->B, p->Hkv, p->Tmax};
  if (!rc) rc = check_apart(kv_strides, cached, 3, p->d, "kv_strides");
  if (!rc) rc = check_visible_all({{seq_lens, "seq_lens"}, {K, "K"}, {V, "V"}});
  if (rc) return rc;
  lod::AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  if (q) {
    a.qb = q_strides[0], a.qh = q_strides[1], a.qt = q_strides[2];
    a.ob = q_out_strides[0], a.oh = q_out_strides[1], a.ot = q_out_strides[2];
  }
  a.kb = kv_new_strides[0], a.kh = kv_new_strides[1], a.kt = kv_new_strides[2];
  a.Hq = q ? p->Hq : 0;
  a.Hkv = p->Hkv;
  a.use_rope = 1;
  a.rope = rope_view(rope);
  a.N = N;
  a.K = K;
  a.V = V;
  a.sb = kv_strides[0], a.sh = kv_strides[1], a.st = kv_strides[2];
  a.Tmax = p->Tmax;
  a.n_new = n_new;
  a.seq_lens = seq_lens;
  const cudaError_t e = lod::launch_append_rows(a, p->dtype, p->d, false, 0, (cudaStream_t)stream);
  return e != cudaSuccess ? cuda_fail(e, "append launch") : ok();
}

int32_t lod_pool_append(const lod_pool* pool, const lod_batch* batch, const lod_rope* rope, const void* q,
                        const int64_t q_strides[2], const void* k, const void* v, const int64_t kv_new_strides[2],
                        void* q_out, const int64_t q_out_strides[2], uint32_t* status, lod_stream_t stream) {
  int32_t rc = check_pool(pool);
  if (!rc) rc = check_batch(pool, batch, true);
  if (rc) return rc;
  const int64_t elem = elem_of(pool->dtype);
  if (q && !rope) return fail(LOD_EINVAL, "q without rope: the queries would only be copied");
  if (rope) rc = check_rope(rope, pool->d);
  const int64_t rows[2] = {batch->N, pool->Hq};
  if (!rc) rc = check_queries(q, q_strides, q_out, q_out_strides, rows, 2, elem, pool->d);
  if (!rc) rc = check_new_kv(k, v, kv_new_strides, 2, elem);
  if (!rc) rc = check_status(status);
  if (rc) return rc;
  lod::AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  if (q) {
    a.qt = q_strides[0], a.qh = q_strides[1];
    a.ot = q_out_strides[0], a.oh = q_out_strides[1];
  }
  a.kt = kv_new_strides[0], a.kh = kv_new_strides[1];
  a.Hq = q ? pool->Hq : 0;
  a.Hkv = pool->Hkv;
  a.use_rope = rope != nullptr;
  if (rope) a.rope = rope_view(rope);
  a.N = batch->N;
  a.pool = pool_view(pool);
  a.batch = batch_view(batch);
  a.status = status;
  const cudaError_t e = lod::launch_append_rows(a, pool->dtype, pool->d, true, pool->bits, (cudaStream_t)stream);
  return e != cudaSuccess ? cuda_fail(e, "pool append launch") : ok();
}

int32_t lod_pool_read(const lod_pool* pool, const lod_batch* batch, int64_t t_begin, int64_t t_end, void* K, void* V,
                      const int64_t kv_strides[3], uint32_t* status, lod_stream_t stream) {
  int32_t rc = check_pool(pool);
  if (!rc) rc = check_batch(pool, batch, false);
  if (rc) return rc;
  if (t_begin < 0 || t_end <= t_begin || t_end > (int64_t)batch->max_blocks * pool->block)
    return fail(LOD_EINVAL, "token range [%lld, %lld) invalid for sequences of at most %lld", (long long)t_begin,
                (long long)t_end, (long long)batch->max_blocks * pool->block);
  if (!K || !V) return fail(LOD_EINVAL, "K and V must be non-NULL");
  if (!aligned16(K) || !aligned16(V)) return fail(LOD_EINVAL, "K and V must be 16-byte aligned");
  rc = check_strides(kv_strides, 3, elem_of(pool->dtype), "kv_strides");
  if (!rc && kv_strides[2] < pool->d) rc = fail(LOD_EINVAL, "token stride smaller than d");
  const int64_t rows[3] = {batch->B, pool->Hkv, t_end};
  if (!rc) rc = check_apart(kv_strides, rows, 3, pool->d, "kv_strides");
  if (!rc) rc = check_visible_all({{K, "K"}, {V, "V"}});
  if (!rc) rc = check_status(status);
  if (rc) return rc;
  lod::ReadArgs a;
  memset(&a, 0, sizeof(a));
  a.pool = pool_view(pool);
  a.batch = batch_view(batch);
  a.K = K;
  a.V = V;
  a.sb = kv_strides[0], a.sh = kv_strides[1], a.st = kv_strides[2];
  a.t_begin = t_begin;
  a.t_end = t_end;
  a.status = status;
  const cudaError_t e = lod::launch_pool_read(a, pool->dtype, pool->bits, pool->d, (cudaStream_t)stream);
  return e != cudaSuccess ? cuda_fail(e, "pool read launch") : ok();
}

int32_t lod_pool_workspace_bytes(const lod_pool* pool, const lod_batch* batch, size_t* bytes) {
  int32_t rc = check_pool_format(pool);
  if (!rc) rc = check_batch_sizes(pool, batch);
  if (!rc) rc = check_new_rows(pool, batch);
  if (rc) return rc;
  if (!bytes) return fail(LOD_EINVAL, "bytes is NULL");
  *bytes = shape_of(pool, batch).total;
  return ok();
}

int32_t lod_pool_attend(const lod_pool* pool, const lod_batch* batch, const void* q, const int64_t q_strides[2],
                        void* out, const int64_t out_strides[2], float* lse, int64_t window, float scale, void* ws,
                        size_t ws_bytes, lod_stream_t stream) {
  int32_t rc = check_pool(pool);
  if (!rc) rc = check_batch(pool, batch, true);
  if (rc) return rc;
  const int64_t elem = elem_of(pool->dtype);
  if (!q || !out) return fail(LOD_EINVAL, "q and out must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(LOD_EINVAL, "q and out must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(LOD_EINVAL, "lse must be 4-byte aligned");
  rc = check_strides(q_strides, 2, elem, "q_strides");
  if (!rc) rc = check_strides(out_strides, 2, elem, "out_strides");
  const int64_t rows[2] = {batch->N, pool->Hq};
  if (!rc) rc = check_apart(out_strides, rows, 2, pool->d, "out_strides");
  if (rc) return rc;
  if (window < 0) return fail(LOD_EINVAL, "window = %lld must be >= 0 (0: none)", (long long)window);
  if (!(scale <= 0.f) && !std::isfinite(scale)) return fail(LOD_EINVAL, "scale must be finite");
  const lod::PoolShape s = shape_of(pool, batch);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < s.total)
    return fail(LOD_EINVAL, "workspace too small (%zu < %zu) or misaligned", ws_bytes, s.total);
  rc = check_visible_all({{q, "q"}, {out, "out"}, {lse, "lse"}, {ws, "workspace"}});
  if (rc) return rc;
  lod::PoolAttendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.qt = q_strides[0], a.qh = q_strides[1];
  a.ot = out_strides[0], a.oh = out_strides[1];
  a.pool = pool_view(pool);
  a.batch = batch_view(batch);
  a.Hq = pool->Hq;
  a.G = pool->Hq / pool->Hkv;
  a.window = window;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)pool->d)) * 1.4426950408889634f;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.planned = !s.inline_plan;
  if (a.planned) {
    a.Wb = reinterpret_cast<int64_t*>(w + s.off_plan);
    a.RT = reinterpret_cast<int32_t*>(a.Wb + batch->B + 1);
    a.pre = a.RT + batch->B + 1;
    if (s.kind == 1) a.rounds = reinterpret_cast<int32_t*>(w + s.off_ml) - 4;  // the plan's last 16 bytes
  }
  a.ml = reinterpret_cast<float2*>(w + s.off_ml);
  a.rec = reinterpret_cast<lod::MergeRec*>(w + s.off_rec);
  a.part = reinterpret_cast<float*>(w + s.off_part);
  a.ctas = s.ctas;
  a.max_rounds = s.max_rounds;
  a.row_bytes = lod::pool_row_bytes(pool->dtype, pool->bits, pool->d);
  lod::PoolMaps maps;
  const bool tma = s.kind != 0 && pool->bits == 0;
  if (tma) {
    const cuuint64_t dims[2] = {(cuuint64_t)pool->d, (cuuint64_t)(pool->blocks * pool->Hkv * pool->block)};
    const cuuint64_t row[1] = {(cuuint64_t)pool->d * 2};
    rc = encode_map(&maps.K, pool->K, 2, dims, row, pool->block);
    if (!rc) rc = encode_map(&maps.V, pool->V, 2, dims, row, pool->block);
    if (rc) return rc;
  }
  const cudaError_t e = lod::launch_pool_attend(a, s, tma ? &maps : nullptr, pool->dtype, pool->bits, pool->d, (cudaStream_t)stream);
  return e != cudaSuccess ? cuda_fail(e, "pool attend launch") : ok();
}

}  // extern "C"
