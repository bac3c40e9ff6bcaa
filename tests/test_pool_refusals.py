"""Argument checks of the projections' append and of the block pool, on the CPU: every call here is refused before
anything reaches a GPU (a pointer that CUDA does not know is itself refused, so fake addresses are never used)."""
import ctypes

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import _lib, api

FAKE = 1 << 20


def pool(**kw):
    base = dict(dtype=_lib.LOD_DTYPE_BF16, bits=0, Hq=16, Hkv=4, d=128, block=16, blocks=64, K=FAKE, V=FAKE, Ke=None,
                Ve=None)
    base.update(kw)
    return _lib.lod_pool(*[base[f] for f, _ in _lib.lod_pool._fields_])


def batch(**kw):
    base = dict(B=2, max_blocks=8, N=5, max_new=3, block_table=FAKE, seq_lens=FAKE, new_begin=FAKE)
    base.update(kw)
    return _lib.lod_batch(*[base[f] for f, _ in _lib.lod_batch._fields_])


def rope(**kw):
    base = dict(q_norm=None, k_norm=None, inv_freq=FAKE, eps=1e-6, rot=128, interleaved=0, pad=0)
    base.update(kw)
    return _lib.lod_rope(*[base[f] for f, _ in _lib.lod_rope._fields_])


def err():
    return _lib.load().lod_last_error().decode()


def s2(a=2048, b=128):
    return (ctypes.c_int64 * 2)(a, b)


def s3(a=1 << 20, b=1 << 16, c=128):
    return (ctypes.c_int64 * 3)(a, b, c)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(_lib.lod_rope) == 40 and _lib.lod_rope.eps.offset == 24
    assert ctypes.sizeof(_lib.lod_pool) == 64 and _lib.lod_pool.blocks.offset == 24
    assert ctypes.sizeof(_lib.lod_batch) == 48 and _lib.lod_batch.N.offset == 8


@pytest.mark.parametrize("kw, code, word", [
    (dict(dtype=2), _lib.LOD_EUNSUPPORTED, "dtype"),
    (dict(bits=4), _lib.LOD_EUNSUPPORTED, "bits"),
    (dict(d=96), _lib.LOD_EUNSUPPORTED, "d = 96"),
    (dict(Hkv=0), _lib.LOD_EINVAL, "Hkv"),
    (dict(Hq=18), _lib.LOD_EINVAL, "multiple"),
    (dict(Hq=65 * 4), _lib.LOD_EUNSUPPORTED, "exceeds 64"),
    (dict(block=8), _lib.LOD_EUNSUPPORTED, "block"),
    (dict(block=48), _lib.LOD_EUNSUPPORTED, "block"),
    (dict(block=256), _lib.LOD_EUNSUPPORTED, "block"),
    (dict(blocks=0), _lib.LOD_EINVAL, "block"),
    (dict(blocks=1 << 25), _lib.LOD_EUNSUPPORTED, "2^31"),
])
def test_bad_pools_are_refused(kw, code, word):
    n = ctypes.c_size_t()
    assert _lib.load().lod_pool_workspace_bytes(ctypes.byref(pool(**kw)), ctypes.byref(batch()), ctypes.byref(n)) == code
    assert word in err()


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=65536), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(N=0),
                                dict(N=1 << 28), dict(max_new=0), dict(max_new=6)])
def test_bad_batches_are_refused(kw):
    n = ctypes.c_size_t()
    rc = _lib.load().lod_pool_workspace_bytes(ctypes.byref(pool()), ctypes.byref(batch(**kw)), ctypes.byref(n))
    assert rc == _lib.LOD_EINVAL and "batch" in err()


def test_calls_of_too_many_tiles_are_refused():
    n = ctypes.c_size_t()
    big = batch(B=1, max_blocks=1 << 26, N=1 << 22, max_new=1 << 22)
    rc = _lib.load().lod_pool_workspace_bytes(ctypes.byref(pool()), ctypes.byref(big), ctypes.byref(n))
    assert rc == _lib.LOD_EUNSUPPORTED and "tiles" in err()
    long = batch(B=1, max_blocks=1 << 16, N=1 << 17, max_new=1 << 15)   # 32K new tokens of a 1M-token sequence
    assert _lib.load().lod_pool_workspace_bytes(ctypes.byref(pool()), ctypes.byref(long), ctypes.byref(n)) == 0


def test_workspace_bytes_need_no_pointers_and_grow():
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    L = _lib.load()
    bare = dict(block_table=None, seq_lens=None, new_begin=None)
    assert L.lod_pool_workspace_bytes(ctypes.byref(pool(K=None, V=None)), ctypes.byref(batch(**bare)), ctypes.byref(n)) == 0
    assert L.lod_pool_workspace_bytes(ctypes.byref(pool()), ctypes.byref(batch(N=100000, max_new=90000)), ctypes.byref(m)) == 0
    assert m.value > n.value > 256
    assert L.lod_pool_workspace_bytes(None, ctypes.byref(batch()), ctypes.byref(n)) == _lib.LOD_EINVAL
    assert L.lod_pool_workspace_bytes(ctypes.byref(pool()), None, ctypes.byref(n)) == _lib.LOD_EINVAL
    assert L.lod_pool_workspace_bytes(ctypes.byref(pool()), ctypes.byref(batch()), None) == _lib.LOD_EINVAL


@pytest.mark.parametrize("kw, word", [
    (dict(K=None), "K and V"), (dict(V=FAKE + 8), "aligned"), (dict(bits=8), "Ke"),
])
def test_pool_pointers_are_checked(kw, word):
    L = _lib.load()
    rc = L.lod_pool_attend(ctypes.byref(pool(**kw)), ctypes.byref(batch()), FAKE, s2(), FAKE, s2(), None, 0, 0.0, FAKE,
                           1 << 30, None)
    assert rc == _lib.LOD_EINVAL and word in err()
    rc = L.lod_pool_read(ctypes.byref(pool(**kw)), ctypes.byref(batch()), 0, 16, FAKE, FAKE, s3(), None, None)
    assert rc == _lib.LOD_EINVAL and word in err()


def test_pointers_that_cuda_does_not_know_are_refused():
    """Without a GPU every address is unknown; with one a made-up address is pageable host memory to CUDA."""
    L = _lib.load()
    rc = L.lod_pool_attend(ctypes.byref(pool()), ctypes.byref(batch()), FAKE, s2(), FAKE, s2(), None, 0, 0.0, FAKE,
                           1 << 30, None)
    assert rc == _lib.LOD_EINVAL and "pool K" in err()
    p = lod.Params(B=2, Hq=16, Hkv=4, d=128, Tmax=4096).c()
    rc = L.lod_append_rope(ctypes.byref(p), ctypes.byref(rope()), None, None, FAKE, FAKE, s3(), 1, FAKE, FAKE, s3(),
                           FAKE, None, None, None)
    assert rc == _lib.LOD_EINVAL and "inv_freq" in err()


@pytest.mark.parametrize("kw, word", [
    (dict(rot=130), "rot"), (dict(rot=-2), "rot"), (dict(rot=7), "rot"), (dict(interleaved=2), "interleaved"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(inv_freq=None), "inv_freq"),
    (dict(inv_freq=FAKE + 2), "inv_freq"), (dict(q_norm=FAKE + 4), "norm"),
])
def test_bad_ropes_are_refused(kw, word):
    L = _lib.load()
    p = lod.Params(B=2, Hq=16, Hkv=4, d=128, Tmax=4096).c()
    rc = L.lod_append_rope(ctypes.byref(p), ctypes.byref(rope(**kw)), None, None, FAKE, FAKE, s3(), 1, FAKE, FAKE,
                           s3(), FAKE, None, None, None)
    assert rc == _lib.LOD_EINVAL and word in err()


def _append(**kw):
    a = dict(p=lod.Params(B=2, Hq=16, Hkv=4, d=128, Tmax=4096).c(), r=rope(rot=0, inv_freq=None), q=None, qs=None, k=FAKE, v=FAKE,
             ks=s3(), n=1, K=FAKE, V=FAKE, st=s3(), lens=FAKE, qo=None, os=None)
    a.update(kw)
    r = None if a["r"] is None else ctypes.byref(a["r"])
    return _lib.load().lod_append_rope(ctypes.byref(a["p"]), r, a["q"], a["qs"], a["k"], a["v"], a["ks"], a["n"], a["K"],
                                       a["V"], a["st"], a["lens"], a["qo"], a["os"], None)


@pytest.mark.parametrize("kw, word", [
    (dict(r=None), "rope"), (dict(lens=None), "seq_lens"), (dict(n=0), "n_new"), (dict(n=4097), "n_new"),
    (dict(k=None), "k and v"), (dict(v=FAKE + 8), "aligned"), (dict(ks=s3(c=4)), "kv_new_strides"),
    (dict(ks=s3(a=-1024)), "kv_new_strides"), (dict(ks=None), "kv_new_strides"), (dict(q=FAKE), "go together"),
    (dict(qo=FAKE), "go together"), (dict(q=FAKE, qo=FAKE + 16, qs=s3(), os=None), "q_out_strides"),
    (dict(q=FAKE, qo=FAKE, qs=s3(), os=s3(b=1 << 15)), "itself"), (dict(K=None), "K, V"),
    (dict(st=s3(c=64)), "stride"),
])
def test_bad_appends_are_refused(kw, word):
    assert _append(**kw) == _lib.LOD_EINVAL and word in err()


def test_unsupported_sizes_of_append_are_refused():
    big = lod.Params(B=1 << 14, Hq=16, Hkv=4, d=128, Tmax=1 << 18).c()
    assert _append(p=big, n=1 << 18) == _lib.LOD_EUNSUPPORTED and "2^31" in err()
    assert _append(p=lod.Params(B=1, Hq=16, Hkv=4, d=96, Tmax=4096).c()) == _lib.LOD_EUNSUPPORTED


# ---- the Python binding's own checks

def test_params_with_a_kept_struct_copy_and_pickle():
    import copy
    import pickle
    p = lod.Params(B=2, Hq=16, Hkv=4, d=128, Tmax=4096)
    assert p.ref() is p.ref()
    for q in (copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and q.ref() is not p.ref()


def _cpu_pool(bits=0, **kw):
    return api.Pool.empty(8, 16, 4, 2, 64, bits=bits, device="cpu", **kw)


def _cpu_batch(tokens=3, max_new=2):
    return api.PoolBatch(torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int64),
                         torch.zeros(3, dtype=torch.int64), tokens=tokens, max_new=max_new)


def test_pool_tensors_are_checked():
    K = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    E = torch.zeros(8, 2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.Pool(K, K[:4], Hq=4, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        api.Pool(K, K, Hq=4, dtype=torch.float32)
    with pytest.raises(TypeError):
        api.Pool(K, K, E, E, Hq=4, dtype=torch.bfloat16)          # codes must be bytes
    with pytest.raises(ValueError):
        api.Pool(K.to(torch.uint8), K.to(torch.uint8), E, E[:, :1], Hq=4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.Pool(K.to(torch.uint8), K.to(torch.uint8), E, None, Hq=4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.Pool(K.transpose(1, 2), K.transpose(1, 2), Hq=4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.Pool.empty(8, 16, 4, 2, 64, bits=4, device="cpu")
    assert _cpu_pool(8).bits == 8 and _cpu_pool().bits == 0


def test_batch_tensors_are_checked():
    t, n, z = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int64)
    for bad in ((t.long(), n, z), (t[:, ::2], n, z), (t, n.int(), z), (t, n[:1], z), (t, n, z[:2]), (t, n, z.int())):
        with pytest.raises(ValueError):
            api.PoolBatch(*bad)


def test_row_shapes_and_types_are_checked():
    p, b = _cpu_pool(), _cpu_batch()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.lod_pool_attend(p, b, q[:2])
    with pytest.raises(ValueError):
        api.lod_pool_attend(p, b, q.float())
    with pytest.raises(ValueError):
        api.lod_pool_attend(p, b, q, out=q[..., :32])
    with pytest.raises(ValueError):
        api.lod_pool_attend(p, b, q, out=q, lse=torch.zeros(3, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        api.lod_pool_append(p, b, k, k[:2])
    with pytest.raises(ValueError):
        api.lod_pool_append(p, b, k, torch.zeros(2, 3, 64, dtype=torch.bfloat16).transpose(0, 1))
    with pytest.raises(ValueError):
        api.lod_pool_append(p, b, k, k, q_out=q)
    with pytest.raises(ValueError):
        api.Rope(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        api.lod_pool_append(p, b, k, k, rope=api.Rope(torch.zeros(32), k_norm=torch.ones(64)))  # fp32 weights, bf16 rows
    with pytest.raises(ValueError):
        api.lod_pool_read(p, b, torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16), 0, 64)
    with pytest.raises(TypeError):
        api.lod_pool_read(p, b, torch.zeros(2, 2, 32, 64), torch.zeros(2, 2, 32, 64))
    with pytest.raises(ValueError):
        api.lod_pool_append(p, api.PoolBatch(b.block_table, b.seq_lens, tokens=3), k, k)


def test_host_tensors_are_refused_by_the_library():
    p, b = _cpu_pool(), _cpu_batch()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((lod.LodError, RuntimeError)):
        api.lod_pool_attend(p, b, q, out=q, ws=torch.zeros(1 << 22, dtype=torch.uint8))
