"""Arguments of the projections' append and of the block pool that the kernels would misread, refused on the CPU."""
import ctypes

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import _lib, api
from tests.test_pool_refusals import FAKE, _append, _cpu_batch, _cpu_pool, err


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
