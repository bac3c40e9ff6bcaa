"""Python binding of the LoD attention library (torch tensors in, C ABI out).

Same names as the C entry points.  PyTorch provides device memory and the
current stream; the binding only checks shapes, allocates outputs and passes
pointers.  All arithmetic runs in liblod.so.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache

import torch

from . import _lib
from ._lib import check, load

_DT = {torch.float32: _lib.LOD_DTYPE_F32, torch.bfloat16: _lib.LOD_DTYPE_BF16}


@dataclass(frozen=True)
class Params:
    """Mirror of lod_params (include/lod.h)."""
    B: int
    Hq: int
    Hkv: int
    d: int
    Tmax: int
    dtype: torch.dtype = torch.bfloat16
    clusters: int = 4
    kmeans_iters: int = 8
    top_groups: int = 8
    top_pages: int = 2
    window: int = 512
    sinks: int = 4
    seed: int = 0
    scale: float = 0.0
    chunk: int = 256
    page: int = 16
    kv_bits: int = 0   # 4: three-tier INT4 (opened pages read from 4-bit codes)
    head_shard: int = 0  # (model KV heads << 16) | first KV head, for a head-sharded process

    def c(self) -> _lib.lod_params:
        return _lib.lod_params(
            _DT[self.dtype], self.B, self.Hq, self.Hkv, self.d, self.chunk, self.page,
            self.clusters, self.kmeans_iters, self.top_groups, self.top_pages, self.window,
            self.sinks, self.kv_bits, self.seed & (2**64 - 1), self.scale, self.head_shard, self.Tmax)

    def ref(self):
        """A reference to the C struct, kept (the fields are frozen)."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r

    def __getstate__(self):  # (copies and pickles leave the reference behind)
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}

    @property
    def page_slots(self) -> int:
        return self.chunk // self.page + self.clusters

    @property
    def g(self) -> int:
        return self.Hq // self.Hkv


class Index:
    """The sixteen device arrays of lod_index, as torch tensors (the arrays
    the parameters do not use are empty)."""

    def __init__(self, params: Params, device="cuda"):
        lib = load()
        sizes = (ctypes.c_size_t * len(_lib.INDEX_FIELDS))()
        check("lod_index_sizes", lib.lod_index_sizes(ctypes.byref(params.c()), sizes))
        p = params
        Cmax, k, P, d = p.Tmax // p.chunk, p.clusters, p.page_slots, p.d
        u = (p.B, p.Hkv)
        self.gK = torch.zeros(*u, Cmax * k, d, dtype=p.dtype, device=device)
        self.gV = torch.zeros_like(self.gK)
        self.gCnt = torch.zeros(*u, Cmax * k, dtype=torch.int32, device=device)
        self.pK = torch.zeros(*u, Cmax * P, d, dtype=p.dtype, device=device)
        self.pV = torch.zeros_like(self.pK)
        self.pCnt = torch.zeros(*u, Cmax * P, dtype=torch.int32, device=device)
        self.pBeg = torch.zeros(*u, Cmax * P, dtype=torch.int16, device=device)
        self.gPage = torch.zeros(*u, Cmax * (k + 1), dtype=torch.int16, device=device)
        self.perm = torch.full((*u, Cmax * p.chunk), -1, dtype=torch.int16, device=device)
        int4 = p.kv_bits == 4
        self.mK = torch.zeros(*u, 0 if int4 else Cmax * p.chunk, d, dtype=p.dtype, device=device)
        self.mV = torch.zeros_like(self.mK)
        self.gMeta = torch.zeros(*u, Cmax * k, dtype=torch.int32, device=device)
        self.qK = torch.zeros(*u, Cmax * p.chunk if int4 else 0, d // 2, dtype=torch.uint8, device=device)
        self.qV = torch.zeros_like(self.qK)
        self.qKs = torch.zeros(*u, Cmax * P if int4 else 0, d, 2, dtype=torch.float32, device=device)
        self.qVs = torch.zeros_like(self.qKs)
        for i, f in enumerate(_lib.INDEX_FIELDS):
            t = getattr(self, f)
            assert t.numel() * t.element_size() == sizes[i], (f, t.numel() * t.element_size(), sizes[i])

    def c(self) -> _lib.lod_index:
        return _lib.lod_index(*[getattr(self, f).data_ptr() for f in _lib.INDEX_FIELDS])

    def nbytes(self) -> int:
        return sum(getattr(self, f).numel() * getattr(self, f).element_size() for f in _lib.INDEX_FIELDS)


def workspace_bytes(params: Params, op: int) -> int:
    n = ctypes.c_size_t()
    check("lod_workspace_bytes", load().lod_workspace_bytes(ctypes.byref(params.c()), op, ctypes.byref(n)))
    return n.value


def workspace(params: Params, op: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for `op` (LOD_OP_BUILD / _DECODE / _PREFILL)."""
    return torch.zeros(workspace_bytes(params, op), dtype=torch.uint8, device=device)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _kv_strides(params: Params, K: torch.Tensor, V: torch.Tensor):
    if K.dtype != params.dtype or V.dtype != params.dtype:
        raise TypeError("K/V dtype %s/%s != params dtype %s" % (K.dtype, V.dtype, params.dtype))
    if K.shape != V.shape or K.dim() != 4 or K.shape[:2] != (params.B, params.Hkv) or K.shape[3] != params.d:
        raise ValueError("K, V must be [B, Hkv, T, d]; got %s / %s" % (tuple(K.shape), tuple(V.shape)))
    if K.stride() != V.stride() or K.stride(3) != 1:
        raise ValueError("K and V must share strides with a contiguous last dimension")
    if K.shape[2] < params.Tmax:
        raise ValueError("KV cache holds %d tokens < Tmax %d" % (K.shape[2], params.Tmax))
    return (ctypes.c_int64 * 3)(K.stride(0), K.stride(1), K.stride(2))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _made_on(stream):
    """Where a call makes the buffers that its caller left out: on the stream that uses them, so that their zero fill
    comes before the kernels and their memory is not handed out again while those run."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def _check_lens(seq_lens, B: int):
    """The kernels read B int64 values in a row: an expanded or strided view would give them others."""
    if seq_lens.shape != (B,) or seq_lens.dtype is not torch.int64 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int64 [B] tensor")


def lod_build_index(params: Params, K, V, chunk_begin: int, chunk_end: int, index: Index, ws=None,
                    stream=None) -> None:
    """Build chunks [chunk_begin, chunk_end) of every (b, kvh) sequence."""
    lib = load()
    st = _kv_strides(params, K, V)
    if ws is None:
        with _made_on(stream):
            ws = workspace(params, _lib.LOD_OP_BUILD, K.device)
    check("lod_build_index", lib.lod_build_index(
        ctypes.byref(params.c()), _ptr(K), _ptr(V), st, chunk_begin, chunk_end,
        ctypes.byref(index.c()), _ptr(ws), ws.numel(), _stream(stream)))


def lod_append_kv(params: Params, K, V, seq_lens, k_new, v_new, stream=None) -> None:
    """Write the current token's key/value rows k_new, v_new ([B, Hkv, d],
    cache dtype; on the device or in pinned host memory, which the kernel
    reads directly) into K/V at positions seq_lens - 1 (one kernel)."""
    lib = load()
    st = _kv_strides(params, K, V)
    shape = (params.B, params.Hkv, params.d)
    for t in (k_new, v_new):
        if t.shape != shape or t.dtype != params.dtype or not t.is_contiguous():
            raise ValueError("k_new / v_new must be contiguous %s %s" % (shape, params.dtype))
    _check_lens(seq_lens, params.B)
    check("lod_append_kv", lib.lod_append_kv(
        ctypes.byref(params.c()), _ptr(K), _ptr(V), st, _ptr(seq_lens), _ptr(k_new), _ptr(v_new),
        _stream(stream)))


def lod_build_ready(params: Params, K, V, seq_lens, index: Index, ws=None, stream=None) -> None:
    """Online build: for every sequence whose length (seq_lens, device int64
    [B]) is a positive multiple of the chunk, build the chunk it just
    completed; the decision is taken on the device, so this can be issued
    every decode step, e.g. on a second stream."""
    lib = load()
    st = _kv_strides(params, K, V)
    _check_lens(seq_lens, params.B)
    if seq_lens.device != K.device:
        raise ValueError("seq_lens must be int64 [B] on the cache's device")
    if ws is None:
        with _made_on(stream):
            ws = workspace(params, _lib.LOD_OP_BUILD, K.device)
    check("lod_build_ready", lib.lod_build_ready(
        ctypes.byref(params.c()), _ptr(K), _ptr(V), st, _ptr(seq_lens), ctypes.byref(index.c()),
        _ptr(ws), ws.numel(), _stream(stream)))


def lod_decode(params: Params, q, K, V, seq_lens, index: Index, out=None, lse=None, sel_groups=None,
               sel_pages=None, ws=None, stream=None):
    """One decode step: q [B, Hq, d] at positions seq_lens - 1.  Returns out.

    q and out may be pinned host tensors: the kernels then read q and store
    out over the host link themselves (no separate copy)."""
    lib = load()
    st = _kv_strides(params, K, V)
    if q.shape != (params.B, params.Hq, params.d) or q.dtype != params.dtype or not q.is_contiguous():
        raise ValueError("q must be contiguous [B, Hq, d] of the cache dtype")
    _check_lens(seq_lens, params.B)
    if not seq_lens.is_cuda:
        raise ValueError("seq_lens must be a device int64 tensor [B]")
    if out is None:
        with _made_on(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=K.device)
    if ws is None:
        with _made_on(stream):
            ws = workspace(params, _lib.LOD_OP_DECODE, K.device)
    check("lod_decode", lib.lod_decode(
        ctypes.byref(params.c()), _ptr(q), _ptr(K), _ptr(V), st, _ptr(seq_lens),
        ctypes.byref(index.c()), _ptr(out), _ptr(lse), _ptr(sel_groups), _ptr(sel_pages), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def lod_prefill(params: Params, q, q_begin: int, K, V, index: Index, out=None, lse=None,
                sel_groups=None, sel_pages=None, ws=None, stream=None):
    """Chunked causal prefill of q [B, Hq, Tq, d] at positions [q_begin, q_begin + Tq).
    Builds the index of the chunks completed in that range first.  Returns out."""
    lib = load()
    st = _kv_strides(params, K, V)
    if q.dim() != 4 or q.shape[:2] != (params.B, params.Hq) or q.shape[3] != params.d \
            or q.dtype != params.dtype or not q.is_contiguous():
        raise ValueError("q must be contiguous [B, Hq, Tq, d] of the cache dtype")
    if out is None:
        with _made_on(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=K.device)
    if ws is None:
        with _made_on(stream):
            ws = workspace(params, _lib.LOD_OP_PREFILL, K.device)
    check("lod_prefill", lib.lod_prefill(
        ctypes.byref(params.c()), _ptr(q), q_begin, q.shape[2], _ptr(K), _ptr(V), st,
        ctypes.byref(index.c()), _ptr(out), _ptr(lse), _ptr(sel_groups), _ptr(sel_pages), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


# ---------------------------------------------------------------- projections into a cache, block pool

# The calls below are made once a layer and token, for a few microseconds of GPU
# work each: their structs, stride arrays and references are built once.

@lru_cache(maxsize=1024)
def _strides(st: tuple):
    """Element strides as the C array (read only)."""
    return (ctypes.c_int64 * len(st))(*st)


class _Fixed:
    """Its attributes stay as they were made: the C struct is filled from them once, and the calls' checks read them."""

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__ and name in self.__dict__:
            raise AttributeError("%s.%s is fixed; make another %s" % (type(self).__name__, name, type(self).__name__))
        super().__setattr__(name, value)


class Rope(_Fixed):
    """Norm and rotation of query and key rows (lod_rope).  inv_freq: float32 [rot / 2] on the device (None: no
    rotation); q_norm, k_norm: [d] weights of the rows' dtype (None: no norm of those rows)."""

    def __init__(self, inv_freq=None, q_norm=None, k_norm=None, interleaved: bool = False, eps: float = 1e-6):
        if inv_freq is not None and (inv_freq.dtype != torch.float32 or inv_freq.dim() != 1
                                     or not inv_freq.is_contiguous()):
            raise ValueError("inv_freq must be a contiguous float32 [rot / 2] tensor")
        for w in (q_norm, k_norm):
            if w is not None and (w.dim() != 1 or not w.is_contiguous()):
                raise ValueError("norm weights must be contiguous [d] tensors")
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm
        self._c = _lib.lod_rope(_addr(q_norm), _addr(k_norm), _addr(inv_freq), eps,
                                0 if inv_freq is None else 2 * inv_freq.numel(), int(interleaved), 0)
        self._fits = [None]  # the (d, dtype) the weights were last checked against
        self._ref = ctypes.byref(self._c)

    def ref(self, d: int, dtype: torch.dtype):
        """The C struct, after checking the weights against the rows they are for."""
        if self._fits[0] != (d, dtype):
            for w in (self.q_norm, self.k_norm):
                if w is not None and (w.shape[0] != d or w.dtype != dtype):
                    raise ValueError("norm weights must be [%d] %s" % (d, dtype))
            self._fits[0] = (d, dtype)
        return self._ref


class Pool(_Fixed):
    """A block pool (lod_pool) over the caller's tensors: K, V [blocks, Hkv, block, d] in dtype, or with Ke, Ve
    (uint8 [blocks, Hkv, block]) as e4m3 codes (float8_e4m3fn or uint8)."""

    def __init__(self, K, V, Ke=None, Ve=None, *, Hq: int, dtype: torch.dtype):
        if K.dim() != 4 or K.shape != V.shape or K.dtype != V.dtype or not K.is_contiguous() or not V.is_contiguous():
            raise ValueError("pool K and V must be contiguous [blocks, Hkv, block, d] of one dtype")
        if (Ke is None) != (Ve is None):
            raise ValueError("Ke and Ve go together")
        if Ke is None:
            if K.dtype != dtype:
                raise TypeError("pool dtype %s != %s (8-bit codes need Ke and Ve)" % (K.dtype, dtype))
        else:
            if K.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError("8-bit codes must be float8_e4m3fn or uint8, not %s" % K.dtype)
            for e in (Ke, Ve):
                if e.shape != K.shape[:3] or e.dtype != torch.uint8 or not e.is_contiguous():
                    raise ValueError("Ke and Ve must be contiguous uint8 [blocks, Hkv, block]")
        self.K, self.V, self.Ke, self.Ve, self.dtype, self.Hq = K, V, Ke, Ve, dtype, Hq
        blocks, self.Hkv, self.block, self.d = K.shape
        self.device = K.device
        self._c = _lib.lod_pool(_DT[dtype], 0 if Ke is None else 8, Hq, self.Hkv, self.d, self.block, blocks,
                                _addr(K), _addr(V), _addr(Ke), _addr(Ve))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, blocks: int, block: int, Hq: int, Hkv: int, d: int, dtype: torch.dtype = torch.bfloat16,
              bits: int = 0, device="cuda") -> "Pool":
        """A zero-filled pool of its own."""
        if bits not in (0, 8):
            raise ValueError("pool bits must be 0 or 8")
        shape = (blocks, Hkv, block, d)
        K = torch.zeros(shape, dtype=torch.uint8 if bits else dtype, device=device)
        e = (lambda: torch.zeros(shape[:3], dtype=torch.uint8, device=device)) if bits else (lambda: None)
        return cls(K, torch.zeros_like(K), e(), e(), Hq=Hq, dtype=dtype)

    @property
    def bits(self) -> int:
        return self._c.bits


class PoolBatch(_Fixed):
    """The sequences of a call (lod_batch): block_table int32 [B, max_blocks], seq_lens int64 [B], new_begin int64
    [B + 1], all on the device; tokens: packed rows N of the call; max_new: most new tokens of one sequence."""

    def __init__(self, block_table, seq_lens, new_begin=None, tokens: int = 1, max_new: int = 1):
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [B, max_blocks] tensor")
        B = block_table.shape[0]
        if seq_lens.shape != (B,) or seq_lens.dtype != torch.int64 or not seq_lens.is_contiguous():
            raise ValueError("seq_lens must be a contiguous int64 [B] tensor")
        if new_begin is not None and (new_begin.shape != (B + 1,) or new_begin.dtype != torch.int64
                                      or not new_begin.is_contiguous()):
            raise ValueError("new_begin must be a contiguous int64 [B + 1] tensor")
        self.block_table, self.seq_lens, self.new_begin = block_table, seq_lens, new_begin
        self.tokens, self.max_new, self.B, self.max_blocks = tokens, max_new, B, block_table.shape[1]
        self._c = _lib.lod_batch(B, block_table.shape[1], tokens, max_new, _addr(block_table), _addr(seq_lens),
                                 _addr(new_begin))
        self._ref = ctypes.byref(self._c)


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(t, shape, dtype, name):
    """Strides of rows with contiguous channels (all dimensions but the last), as the C array."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s must be %s %s; got %s %s" % (name, shape, dtype, tuple(t.shape), t.dtype))
    st = t.stride()
    if st[-1] != 1:
        raise ValueError("%s must have contiguous channels" % name)
    return _strides(st[:-1])


def _stream_handle(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if device.type != "cuda":
        raise RuntimeError("the cache must be on a CUDA device, not %s" % device)
    return torch._C._cuda_getCurrentRawStream(device.index)  # (torch.cuda.current_stream builds an object: 3 us)


def _status_word(status):
    if status is not None and (status.numel() < 1 or status.element_size() != 4):
        raise ValueError("status must be a 4-byte integer tensor")
    return _addr(status)


def lod_append_rope(params: Params, rope: Rope, q, k, v, K, V, seq_lens, q_out=None, stream=None):
    """Append the newest tokens' projections to the dense cache: k, v [B, Hkv, n, d] go to positions
    [seq_lens - n, seq_lens) of K, V, the keys normed and rotated by `rope`, and the normed and rotated q
    [B, Hq, n, d] to q_out (which may be q).  q, k, v may be strided views of one fused projection; q None
    appends the keys and values alone.  Returns q_out."""
    B, Hkv, d, dt = params.B, params.Hkv, params.d, params.dtype
    st = K.stride()
    if K.dtype is not dt or V.dtype is not dt or K.shape != V.shape or V.stride() != st or len(st) != 4 \
            or st[3] != 1 or K.shape[0] != B or K.shape[1] != Hkv or K.shape[3] != d or K.shape[2] < params.Tmax:
        _kv_strides(params, K, V)  # names what is wrong
    n = k.shape[2] if k.dim() == 4 else -1
    ks = _rows(k, (B, Hkv, n, d), dt, "k")
    if _rows(v, (B, Hkv, n, d), dt, "v") is not ks and v.stride() != k.stride():
        raise ValueError("k and v must share strides")
    _check_lens(seq_lens, B)
    qs = os = None
    if q is not None:
        shape = (B, params.Hq, n, d)
        qs = _rows(q, shape, dt, "q")
        if q_out is None:
            with _made_on(stream):
                q_out = torch.empty(shape, dtype=dt, device=K.device)
        os = _rows(q_out, shape, dt, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    check("lod_append_rope", load().lod_append_rope(
        params.ref(), rope.ref(d, dt), _addr(q), qs, k.data_ptr(), v.data_ptr(), ks, n, K.data_ptr(), V.data_ptr(),
        _strides(st[:3]), seq_lens.data_ptr(), _addr(q_out), os, _stream_handle(stream, K.device)))
    return q_out


def lod_pool_append(pool: Pool, batch: PoolBatch, k, v, rope: Rope | None = None, q=None, q_out=None, status=None,
                    stream=None):
    """Write the new tokens' k, v [N, Hkv, d] into the pool, in its format and normed and rotated by `rope`, and
    with q [N, Hq, d] the normed and rotated queries to q_out (which may be q).  Returns q_out."""
    if batch.new_begin is None:
        raise ValueError("the batch has no new_begin")
    N, d, dt = batch.tokens, pool.d, pool.dtype
    ks = _rows(k, (N, pool.Hkv, d), dt, "k")
    if _rows(v, (N, pool.Hkv, d), dt, "v") is not ks and v.stride() != k.stride():
        raise ValueError("k and v must share strides")
    qs = os = None
    if q is not None:
        qs = _rows(q, (N, pool.Hq, d), dt, "q")
        if q_out is None:
            with _made_on(stream):
                q_out = torch.empty(N, pool.Hq, d, dtype=dt, device=pool.K.device)
        os = _rows(q_out, (N, pool.Hq, d), dt, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    check("lod_pool_append", load().lod_pool_append(
        pool._ref, batch._ref, None if rope is None else rope.ref(d, dt), _addr(q), qs, k.data_ptr(), v.data_ptr(),
        ks, _addr(q_out), os, _status_word(status), _stream_handle(stream, pool.device)))
    return q_out


def lod_pool_read(pool: Pool, batch: PoolBatch, K, V, t_begin: int = 0, t_end: int | None = None, status=None,
                  stream=None) -> None:
    """Read tokens [t_begin, min(t_end, seq_lens)) of every sequence into the dense cache K, V [B, Hkv, T, d] of
    the pool's dtype (t_end None: up to T)."""
    shape, st = K.shape, K.stride()
    if len(st) != 4 or shape[0] != batch.B or shape[1] != pool.Hkv or shape[3] != pool.d or shape != V.shape:
        raise ValueError("K, V must be [B, Hkv, T, d]; got %s / %s" % (tuple(K.shape), tuple(V.shape)))
    if K.dtype is not pool.dtype or V.dtype is not pool.dtype:
        raise TypeError("K/V dtype %s/%s != pool dtype %s" % (K.dtype, V.dtype, pool.dtype))
    if st != V.stride() or st[3] != 1:
        raise ValueError("K and V must share strides with a contiguous last dimension")
    if t_end is None:
        t_end = min(shape[2], batch.max_blocks * pool.block)
    if t_end > shape[2]:
        raise ValueError("t_end %d behind the dense cache's %d tokens" % (t_end, shape[2]))
    check("lod_pool_read", load().lod_pool_read(
        pool._ref, batch._ref, t_begin, t_end, K.data_ptr(), V.data_ptr(), _strides(st[:3]),
        _status_word(status), _stream_handle(stream, pool.device)))


def pool_workspace_bytes(pool: Pool, batch: PoolBatch) -> int:
    n = ctypes.c_size_t()
    check("lod_pool_workspace_bytes", load().lod_pool_workspace_bytes(pool._ref, batch._ref, ctypes.byref(n)))
    return n.value


def pool_workspace(pool: Pool, batch: PoolBatch) -> torch.Tensor:
    """A zero-filled workspace of lod_pool_attend for this batch."""
    return torch.zeros(pool_workspace_bytes(pool, batch), dtype=torch.uint8, device=pool.K.device)


def lod_pool_attend(pool: Pool, batch: PoolBatch, q, out=None, lse=None, window: int = 0, scale: float = 0.0,
                    ws=None, stream=None):
    """Exact causal attention of the new tokens' q [N, Hq, d] over the pool (which already holds them); window > 0
    limits each query to its last `window` keys; lse float32 [N, Hq].  Returns out.  The status word (refused
    sequences, bad blocks) is the first of `ws`; without ws it is lost with the call's own workspace."""
    if batch.new_begin is None:
        raise ValueError("the batch has no new_begin")
    shape = (batch.tokens, pool.Hq, pool.d)
    qs = _rows(q, shape, pool.dtype, "q")
    if out is None:
        with _made_on(stream):
            out = torch.empty(shape, dtype=pool.dtype, device=pool.device)
    os = _rows(out, shape, pool.dtype, "out")
    if lse is not None and (lse.shape != shape[:2] or lse.dtype is not torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [N, Hq] tensor")
    if ws is None:
        with _made_on(stream):
            ws = pool_workspace(pool, batch)
    check("lod_pool_attend", load().lod_pool_attend(
        pool._ref, batch._ref, q.data_ptr(), qs, out.data_ptr(), os, _addr(lse), window, scale, ws.data_ptr(),
        ws.numel() * ws.element_size(), _stream_handle(stream, pool.device)))
    return out


def lod_get_status(ws, stream=None) -> int:
    """Read and clear the device status word (LOD_ST_* bits); synchronises."""
    v = ctypes.c_uint32()
    rc = load().lod_get_status(_ptr(ws), _stream(stream), ctypes.byref(v))
    if rc not in (_lib.LOD_OK, _lib.LOD_EDEVICE):
        check("lod_get_status", rc)
    return v.value
