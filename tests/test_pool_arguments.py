"""Arguments of the projections' append and of the block pool that the kernels would misread, refused on the CPU."""
import ctypes

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import _lib, api
from tests.test_pool_refusals import FAKE, _append, _cpu_batch, _cpu_pool, err, s3


def _dense(B=3, T=256):
    p = lod.Params(B=B, Hq=2, Hkv=1, d=64, Tmax=T, dtype=torch.bfloat16)
    K = torch.zeros(B, 1, T, 64, dtype=torch.bfloat16)
    return p, K, torch.zeros_like(K)


@pytest.mark.parametrize("lens", [
    torch.tensor([5]).expand(3),                       # one length for the batch: one value behind the pointer
    torch.arange(6)[::2],
    torch.arange(6).view(3, 2)[:, 0],
    torch.arange(3, dtype=torch.int32),
    torch.arange(2),
])
def test_lengths_that_are_no_row_of_int64_are_refused(lens):
    p, K, V = _dense()
    k = torch.zeros(3, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="seq_lens"):
        api.lod_append_rope(p, api.Rope(), None, k, k, K, V, lens)
    with pytest.raises(ValueError, match="seq_lens"):
        api.lod_append_kv(p, K, V, lens, k[:, :, 0], k[:, :, 0])
    with pytest.raises(ValueError, match="seq_lens"):
        api.lod_build_ready(p, K, V, lens, None)
    with pytest.raises(ValueError, match="seq_lens"):
        api.lod_decode(p, torch.zeros(3, 2, 64, dtype=torch.bfloat16), K, V, lens, None)


def test_misaligned_lengths_are_refused():
    assert _append(lens=FAKE + 4) == _lib.LOD_EINVAL and "seq_lens" in err()


@pytest.mark.parametrize("name, value", [("tokens", 2), ("max_new", 5), ("B", 1), ("block_table", None), ("seq_lens", None)])
def test_a_batch_is_fixed(name, value):
    """The checks read the attributes and the kernels the C struct: 1 packed row checked, 3 written."""
    b = _cpu_batch()
    with pytest.raises(AttributeError, match=name):
        setattr(b, name, value)
    assert getattr(b, name) is not value and b._c.N == 3


def test_a_pool_and_a_rope_are_fixed():
    p, r = _cpu_pool(), api.Rope(torch.zeros(32))
    for obj, name in ((p, "K"), (p, "Hq"), (p, "d"), (p, "dtype"), (r, "inv_freq"), (r, "q_norm")):
        with pytest.raises(AttributeError, match=name):
            setattr(obj, name, None)
    r.ref(64, torch.bfloat16)
    r.ref(128, torch.float32)


@pytest.mark.parametrize("os, good", [
    (s3(4096 * 16, 128, 16 * 128), True),              # [b][token][head]
    (s3(128, 256, 4096), True),                        # [token][head][b], B = 2 and 16 heads
    (s3(1 << 60, 128, 2048), True),
    (s3(0, 128, 2048), False), (s3(1 << 20, 0, 128), False), (s3(1 << 20, 128, 0), False),
    (s3(1 << 20, 64, 2048), False),                    # heads closer than a row
    (s3(1 << 20, 128, 1024), False),                   # a token's 16 heads reach into the next token
    (s3(2048, 128, 2048), False),
    (s3(1 << 62, 1 << 62, 1 << 62), False),
])
def test_outputs_whose_rows_overlap_are_refused(os, good):
    """2 sequences of 3 tokens, 16 heads of 128 channels.  (Good strides get as far as the made-up addresses.)"""
    rc = _append(q=FAKE, qo=FAKE + 4096, qs=s3(), os=os, n=3)
    assert rc == _lib.LOD_EINVAL and ("overlap" in err()) != good, err()


def test_single_rows_may_have_any_stride():
    p = lod.Params(B=1, Hq=1, Hkv=1, d=128, Tmax=4096).c()
    assert _append(p=p, q=FAKE, qo=FAKE + 4096, qs=s3(), os=s3(0, 0, 0), n=1) == _lib.LOD_EINVAL and "overlap" not in err()
