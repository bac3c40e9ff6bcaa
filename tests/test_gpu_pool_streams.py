"""Calls on a stream of their own that leave their buffers to the binding."""
import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import api
from tests.test_gpu_pool import BF, F32, gen, make_batch, make_pool, make_rope, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def beside(stream, call, sizes):
    """The result of `call` on a stream that is busy, while the current stream takes memory of the given sizes, fills
    it, and must find it as it was."""
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    got = call()
    mine = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    stream.synchronize()
    torch.cuda.synchronize()
    assert all((x == 0x5a).all() for x in mine)
    return got


@pytest.mark.parametrize("n, dtype, bits", [(1, BF, 8), (90, BF, 0), (90, F32, 0)])
def test_pool_calls_on_a_busy_stream_make_their_buffers_there(n, dtype, bits):
    g = gen(301)
    lens = [3000, 700]
    pool, table = make_pool(g, lens, 32, 16, 2, 128, dtype, bits)
    _, batch = make_batch(table, lens, [n, n])
    rope, _ = make_rope(g, 128, dtype, 128, False, True)
    q, k = randn(g, 2 * n, 16, 128, dtype=dtype), randn(g, 2 * n, 2, 128, dtype=dtype)
    ws = api.pool_workspace_bytes(pool, batch)
    size = q.numel() * q.element_size()
    side = torch.cuda.Stream()
    want_q = lod.lod_pool_append(pool, batch, k, k, rope=rope, q=q)
    want = lod.lod_pool_attend(pool, batch, want_q)
    for _ in range(3):
        got_q = beside(side, lambda: lod.lod_pool_append(pool, batch, k, k, rope=rope, q=q, stream=side), [size])
        assert torch.equal(got_q, want_q)
        got = beside(side, lambda: lod.lod_pool_attend(pool, batch, want_q, stream=side), [size, ws])
        assert torch.equal(got, want)


def test_dense_calls_on_a_busy_stream_make_their_buffers_there():
    g = gen(302)
    p = lod.Params(B=2, Hq=8, Hkv=2, d=128, Tmax=1024, dtype=BF)
    rope, _ = make_rope(g, 128, BF, 128, False, True)
    K, V = (randn(g, 2, 2, 1024, 128, dtype=BF) for _ in range(2))
    lens = torch.tensor([900, 1000], device="cuda")
    q, k = randn(g, 2, 8, 5, 128, dtype=BF), randn(g, 2, 2, 5, 128, dtype=BF)
    ix, side = lod.Index(p), torch.cuda.Stream()
    want = lod.lod_append_rope(p, rope, q, k, k, K, V, lens)
    lod.lod_build_index(p, K, V, 0, 3, ix)
    d1 = q[:, :, 0].contiguous()
    want_d = lod.lod_decode(p, d1, K, V, lens, ix)
    want_p = lod.lod_prefill(p, q, 768, K, V, ix)
    sizes = [q.numel() * 2] + [api.workspace_bytes(p, op) for op in (lod.LOD_OP_BUILD, lod.LOD_OP_DECODE, lod.LOD_OP_PREFILL)]
    got = beside(side, lambda: lod.lod_append_rope(p, rope, q, k, k, K, V, lens, stream=side), sizes[:1])
    assert torch.equal(got, want)
    beside(side, lambda: lod.lod_build_index(p, K, V, 0, 3, ix, stream=side), sizes)
    assert torch.equal(beside(side, lambda: lod.lod_decode(p, d1, K, V, lens, ix, stream=side), sizes), want_d)
    assert torch.equal(beside(side, lambda: lod.lod_prefill(p, q, 768, K, V, ix, stream=side), sizes), want_p)
