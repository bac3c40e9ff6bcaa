"""Attention over the block pool at the edges of its number formats, on the GPU: infinite scores, scales that
underflow, value rows of zeros and of very different sizes, NaN in rows that a query does not see."""
import math

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import api
from tests import pooltest as pt
from tests.test_gpu_pool import BF, F32, close, gen, make_batch, randn

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def pool_of(rows, block, Hq, dtype, bits, g):
    """A pool that holds the sequences' rows [(k, v)], each [length, Hkv, d], its blocks dealt out at random."""
    Hkv, d = rows[0][0].shape[1:]
    need = [-(-len(k) // block) for k, _ in rows]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(rows), max(need)), -1, dtype=torch.int32, device="cuda")
    pool = api.Pool.empty(sum(need), block, Hq, Hkv, d, dtype, bits)
    at = 0
    for b, (k, v) in enumerate(rows):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = torch.arange(len(k), device="cuda")
        blk, off = table[b].long()[t // block], t % block
        for X, E, x in ((pool.K, pool.Ke, k), (pool.V, pool.Ve, v)):
            if bits:
                X[blk, :, off], E[blk, :, off] = pt.quantise64(x.to(dtype))
            else:
                X[blk, :, off] = x.to(dtype)
    return pool, table


def attend(pool, table, lens, new, q, window=0, scale=0.0):
    begin, batch = make_batch(table, lens, new)
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    ws = api.pool_workspace(pool, batch)
    lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, window=window, scale=scale, ws=ws)
    return begin, out, lse, lod.lod_get_status(ws)


def check(pool, table, lens, new, q, scale=0.0):
    begin, out, lse, status = attend(pool, table, lens, new, q, scale=scale)
    assert status == 0
    o, z, to, tz = pt.attend64(pool, table, lens, begin, q, 0, scale)
    close(lse, z, tz, "lse")
    close(out, o, to, "out")


# ------------------------------------------------------------------ infinite scores

@pytest.mark.parametrize("dtype, d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("n", [1, 60, 150])
def test_a_key_of_infinite_score_makes_the_row_nan(n, dtype, d):
    """An infinite key channel at each place of a tile's first 32 keys: a query on its positive side has the weight
    inf - inf; on its negative side the key has none."""
    B, L, Hq, Hkv = 32, 128 + n + 9, 4, 2
    g = gen(201)
    rows = [(randn(g, L, Hkv, d), randn(g, L, Hkv, d)) for _ in range(B)]
    at = [b if n == 1 or b % 2 else L - n + b // 2 for b in range(B)]  # among the old keys, or the new ones
    for b in range(B):
        rows[b][0][at[b], :, 3] = math.inf
    pool, table = pool_of(rows, 32, Hq, dtype, 0, g)
    q = randn(g, B * n, Hq, d, dtype=dtype)
    begin, out, lse, status = attend(pool, table, [L] * B, [n] * B, q)
    assert status == 0
    bad = [torch.arange(L, device="cuda") == at[b] for b in range(B)]
    o, z, to, tz = pt.attend64(pool, table, [L] * B, begin, q, bad_keys=bad)
    pos = (torch.arange(n, device="cuda") + L - n).repeat(B)
    sees = pos >= torch.tensor(at, device="cuda").repeat_interleave(n)
    hit = sees[:, None] & (q[..., 3] > 0)
    assert 0.2 < hit.float().mean() < 0.6
    assert torch.isnan(out[hit]).all(), "%d of %d" % (int((~torch.isnan(out[hit])).any(-1).sum()), int(hit.sum()))
    assert torch.isnan(lse[hit]).all()
    close(out[~hit], o[~hit], to[~hit], "out")
    close(lse[~hit], z[~hit], tz[~hit], "lse")


# ------------------------------------------------------------------ scales below fp32's range

@pytest.mark.parametrize("dtype, bits", [(BF, 8), (BF, 0), (F32, 8)])
@pytest.mark.parametrize("n", [1, 60, 300])
@pytest.mark.parametrize("qmul, scale", [(2.0 ** -15, 0.0), (2.0 ** -60, 0.0), (1.0, 1e-30), (2.0 ** -100, 1e-20)])
def test_key_tiles_of_zeros_and_bad_blocks_with_small_queries(qmul, scale, n, dtype, bits):
    """A tile of zero keys has the smallest exponent a row can have; with a small query the product of the scale and
    both powers of two lies below fp32's range."""
    g = gen(202)
    L, Hq, Hkv, d = 520, 4, 2, 64
    k, v = randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    k[128:384] = 0
    pool, table = pool_of([(k, v)], 64, Hq, dtype, bits, g)
    check(pool, table, [L], [n], (randn(g, n, Hq, d) * qmul).to(dtype), scale)
    gone = torch.zeros(L, dtype=torch.bool, device="cuda")
    gone[128:256] = True
    safe = table.clone()
    table[0, 2:4] = -1
    q = (randn(g, n, Hq, d) * qmul).to(dtype)
    begin, out, lse, _ = attend(pool, table, [L], [n], q, scale=scale)
    o, z, to, tz = pt.attend64(pool, safe, [L], begin, q, 0, scale, bad_keys=[gone])
    close(lse, z, tz, "lse")
    close(out, o, to, "out")


# ------------------------------------------------------------------ value rows of very different sizes

def weighted(g, L, Hkv, d, powers):
    """Keys whose scores against the query (1, 0, 0, ...) at scale 1 are powers * ln 2."""
    k = torch.zeros(L, Hkv, d, device="cuda")
    k[..., 0] = powers[:, None] * LN2
    return k


def unit_queries(n, Hq, d, dtype):
    q = torch.zeros(n, Hq, d, dtype=dtype, device="cuda")
    q[..., 0] = 1
    return q


@pytest.mark.parametrize("dtype, bits", [(BF, 8), (BF, 0), (F32, 8)])
@pytest.mark.parametrize("n", [1, 2, 4, 60])
@pytest.mark.parametrize("size", [300.0, 2.0 ** 15, 2.0 ** 40, 2.0 ** -20])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
def test_keys_of_zero_values_keep_their_weight(where, size, n, dtype, bits):
    """Most value rows are zeros; a few are large, and their scores 10 to 14 powers of two above the rest."""
    g = gen(203)
    L, Hq, Hkv, d = 6000, 8, 1, 128
    powers = torch.randn(L, generator=g, device="cuda") - 2
    v = torch.zeros(L, Hkv, d, device="cuda")
    top = {"first": torch.arange(3, 9), "last": torch.arange(L - 70, L - 64), "spread": torch.arange(700, L - 700, 900)}[where]
    powers[top] = 10 + 4 * torch.rand(len(top), generator=g, device="cuda")
    v[top] = size * (1 + 0.4 * torch.rand(len(top), Hkv, d, generator=g, device="cuda"))
    pool, table = pool_of([(weighted(g, L, Hkv, d, powers), v)], 32, Hq, dtype, bits, g)
    check(pool, table, [L], [n], unit_queries(n, Hq, d, dtype), 1.0)


@pytest.mark.parametrize("dtype, bits", [(BF, 8), (BF, 0), (F32, 8)])
@pytest.mark.parametrize("n", [1, 4, 60, 300])
@pytest.mark.parametrize("order", ["large first", "small first", "turns", "rising", "falling"])
@pytest.mark.parametrize("small, large, low", [(2.0 ** -20, 2.0 ** 20, -60.0), (2.0 ** -9, 2.0 ** 9, -40.0),
                                               (2.0 ** -15, 2.0 ** 24, -100.0), (1.0, 2.0 ** 40, -90.0)])
def test_tiles_of_small_values_beside_tiles_of_large_ones(small, large, low, order, n, dtype, bits):
    """Tiles whose values differ by up to 2^40, the large ones of hardly any weight: the outputs are the small ones'."""
    g = gen(204)
    L, Hq, Hkv, d, tile = 1600, 8, 2, 64, 128
    at = torch.arange(L, device="cuda") // tile
    last = int(at[-1])
    frac = {"large first": (at < 3).float(), "small first": ((at >= 5) & (at < 9)).float(), "turns": (at % 2 == 0).float(),
            "rising": at.float() / last, "falling": 1 - at.float() / last}[order]
    frac[L - 301:] = frac[L - 301:] * 0 + float(frac[L - 302])  # (every new token sees both kinds before it)
    powers = low * frac + 0.5 * torch.randn(L, generator=g, device="cuda")
    f = small * (large / small) ** frac.round(decimals=1)
    v = randn(g, L, Hkv, d) * f[:, None, None]
    pool, table = pool_of([(weighted(g, L, Hkv, d, powers), v)], 64, Hq, dtype, bits, g)
    check(pool, table, [L], [n], unit_queries(n, Hq, d, dtype), 1.0)


@pytest.mark.parametrize("dtype, bits", [(BF, 8), (BF, 0), (F32, 8)])
@pytest.mark.parametrize("n", [1, 4, 60])
def test_huge_rows_that_no_query_sees_cost_nothing(n, dtype, bits):
    """The tile in which the window begins also holds rows before it, 2^90 times as large."""
    g = gen(206)
    L, Hq, Hkv, d, window = 1000, 8, 2, 64, 300
    k, v = randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    k[L - n - window - 20:L - n - window - 10] *= 2.0 ** 90
    v[L - n - window - 20:L - n - window - 10] *= 2.0 ** 90
    pool, table = pool_of([(k, v)], 32, Hq, dtype, bits, g)
    q = randn(g, n, Hq, d, dtype=dtype)
    begin, out, lse, status = attend(pool, table, [L], [n], q, window=window)
    assert status == 0
    o, z, to, tz = pt.attend64(pool, table, [L], begin, q, window)
    assert o.abs().max() < 10
    close(lse, z, tz, "lse")
    close(out, o, to, "out")


@pytest.mark.parametrize("dtype, bits", [(BF, 8), (BF, 0), (F32, 8)])
def test_huge_rows_of_later_tokens_cost_earlier_ones_nothing(dtype, bits):
    """Two tokens, 8 apart in one key tile, of 64 heads a KV head: the later one's rows are 2^90 times as large."""
    g = gen(207)
    L, Hq, Hkv, d, n = 128 * 6, 64, 1, 64, 12
    k, v = randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    k[-4:] *= 2.0 ** 90
    v[-4:] *= 2.0 ** 90
    pool, table = pool_of([(k, v)], 32, Hq, dtype, bits, g)
    q = randn(g, n, Hq, d, dtype=dtype)
    begin, out, lse, status = attend(pool, table, [L], [n], q)
    o, z, to, tz = pt.attend64(pool, table, [L], begin, q)
    assert status == 0 and o[:4].abs().max() < 10
    close(lse[:4], z[:4], tz[:4], "lse")
    close(out[:4], o[:4], to[:4], "out")


# ------------------------------------------------------------------ NaN behind a query

@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0), (F32, 8)])
@pytest.mark.parametrize("G, n, T", [(16, 130, 120), (4, 300, 280), (1, 700, 600), (64, 70, 66)])
def test_a_nan_value_reaches_no_queries_far_before_it(G, n, T, dtype, bits):
    """New token T's value row is NaN: queries of its own sequence more than 256 query rows before T's do not see it,
    also where its key shares a tile with theirs."""
    g = gen(205)
    L, Hkv, d = 256 + n, 2, 64
    k, v = randn(g, L, Hkv, d, dtype=dtype), randn(g, L, Hkv, d, dtype=dtype)
    pool, table = pool_of([(k, v)], 32, G * Hkv, dtype, bits, g)
    _, batch = make_batch(table, [L], [n])
    v[L - n + T, :, 5] = math.nan
    lod.lod_pool_append(pool, batch, k[L - n:], v[L - n:])
    q = randn(g, n, G * Hkv, d, dtype=dtype)
    begin, out, lse, status = attend(pool, table, [L], [n], q)
    assert status == 0
    o, z, to, tz = pt.attend64(pool, table, [L], begin, q)
    close(lse, z, tz, "lse")
    far = T - -(-256 // G)
    assert far > 0 and torch.isfinite(o[:far]).all()
    close(out[:far], o[:far], to[:far], "out")
    assert torch.isnan(out[T:, :, 5]).all()
