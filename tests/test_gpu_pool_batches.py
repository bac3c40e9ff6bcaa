"""Batches of the block pool whose new_begin falls, and batches of many sequences, on the GPU: which sequences a call
takes, that no row is given to two, that the workspace is not left, and the values against the 64-bit forms."""
import math

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import api
from tests import pooltest as pt
from tests.test_gpu_pool import BF, F32, ST, close, gen, make_pool, make_rope, randn, rope_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def taken(begin, lens, N, max_new):
    """The sequences of a batch that are not refused, and the rows of [0, N) that only refused ones name."""
    ok, top = [], -math.inf
    for b, L in enumerate(lens):
        r0, r1 = begin[b], begin[b + 1]
        top = max(top, r0)
        ok.append(0 <= r0 <= r1 <= N and r1 - r0 <= min(max_new, L) and (r0 == top or r0 == r1))
    owned, named = set(), set()
    for b in range(len(lens)):
        rows = range(max(begin[b], 0), min(begin[b + 1], N))
        if ok[b]:
            assert owned.isdisjoint(rows)
            owned.update(rows)
        else:
            named.update(rows)
    return ok, sorted(owned), sorted(named - owned)


def walk(begin, lens, N, max_new, Hq, Hkv, d, block, dtype, bits, seed):
    """Append and attention of one batch, checked row by row."""
    B = len(lens)
    ok, owned, cleared = taken(begin, lens, N, max_new)
    g = gen(seed)
    pool, table = make_pool(g, lens, block, Hq, Hkv, d, dtype, bits)
    batch = api.PoolBatch(table, torch.tensor(lens, device="cuda"), torch.tensor(begin, device="cuda"), tokens=N,
                          max_new=max_new)
    q, k, v = randn(g, N, Hq, d, dtype=dtype), randn(g, N, Hkv, d, dtype=dtype), randn(g, N, Hkv, d, dtype=dtype)

    # the append writes the new rows of the sequences that are taken, and nothing else
    want = [None if x is None else x.clone() for x in (pool.K, pool.V, pool.Ke, pool.Ve)]
    for b in range(B):
        if ok[b] and begin[b + 1] > begin[b]:
            n = begin[b + 1] - begin[b]
            t = torch.arange(lens[b] - n, lens[b], device="cuda")
            blk, off = table[b].long()[t // block], t % block
            for X, E, x in ((want[0], want[2], k), (want[1], want[3], v)):
                rows = x[begin[b]:begin[b + 1]]
                if bits:
                    X[blk, :, off], E[blk, :, off] = pt.quantise64(rows)
                else:
                    X[blk, :, off] = rows
    rope = api.Rope()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((N, Hq, d), 9.0, dtype=dtype, device="cuda")
    lod.lod_pool_append(pool, batch, k, v, rope=rope, q=q, q_out=out, status=status)
    assert int(status) == (0 if all(ok) else ST["seqlen"])
    mine = torch.zeros(N, dtype=torch.bool, device="cuda")
    mine[owned] = True
    assert torch.equal(out[mine], q[mine]) and (out[~mine] == 9).all()
    for X, Y in zip((pool.K, pool.V, pool.Ke, pool.Ve), want):
        assert X is None or torch.equal(X.view(torch.uint8), Y.view(torch.uint8))

    # the attention, with a workspace of the size that was asked for and a guard behind it
    need = api.pool_workspace_bytes(pool, batch)
    buf = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    buf[need:] = 0x5a
    out.fill_(9.0)
    lse = torch.full((N, Hq), 9.0, device="cuda")
    lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, ws=buf[:need])
    assert lod.lod_get_status(buf[:need]) == (0 if all(ok) else ST["seqlen"])
    assert (buf[need:] == 0x5a).all()
    gone = torch.zeros(N, dtype=torch.bool, device="cuda")
    gone[cleared] = True
    assert (out[gone] == 0).all() and (lse[gone] == -math.inf).all()
    assert (out[~gone & ~mine] == 9).all() and (lse[~gone & ~mine] == 9).all()
    for b in range(0, B, 1 if B < 100 else 7):
        r0, r1 = begin[b], begin[b + 1]
        if ok[b] and r1 > r0:
            o, z, to, tz = pt.attend64(pool, table[b:b + 1], lens[b:b + 1], [0, r1 - r0], q[r0:r1])
            close(out[r0:r1], o, to, "out %d" % b)
            close(lse[r0:r1], z, tz, "lse %d" % b)


FALLING = [
    ([0, 6, 0, 6], 6),                     # two sequences of the same rows
    ([0, 5, 2, 8, 11], 6),                 # rows 5 .. 7 are named by a refused sequence alone
    ([6, 9, 1, 4, 9, 12], 5),              # rows below the first entry
    ([0, 40, 5, 8, 8, 45, 50], 6),         # a refused one that reaches over others
    ([2, 4, 4, 3, 3, 9, 9], 6),            # empty ones in the fall
    ([0, 3, 1 << 40, 3, 6], 6),
    ([-3, 2, 5, 4, 9], 6),
]


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0)])
@pytest.mark.parametrize("begin, max_new", FALLING)
def test_new_begin_that_falls(begin, max_new, dtype, bits):
    lens = [70 + 13 * b for b in range(len(begin) - 1)]
    walk(begin, lens, 51, max_new, 4, 2, 64, 16, dtype, bits, 101)


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 8)])
@pytest.mark.parametrize("n", [40, 700])
def test_long_sequences_of_the_same_rows(n, dtype, bits):
    """The list holds the row tiles of N rows: a second and third sequence of the same ones would not fit."""
    walk([0, n, 0, n, 0, n, n + 20], [n + 30, n + 5, n + 60, n + 9, n, 90], n + 25, n, 8, 1, 128, 32, dtype, bits, 102)


@pytest.mark.parametrize("dtype, bits", [(BF, 8), (F32, 0)])
@pytest.mark.parametrize("G, B", [(1, 33), (2, 70), (8, 300), (1, 1100), (16, 1060)])
@pytest.mark.parametrize("falls", [False, True])
def test_batches_of_many_sequences(falls, G, B, dtype, bits):
    """More sequences than a warp's probes, than a CTA lays out by itself (256), than a pass of the plan (1024); with
    G = 16 a sequence of 3 new tokens makes 48 rows."""
    g = torch.Generator().manual_seed(B)
    new = torch.randint(0, 4, (B,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 60, (B,), generator=g))]
    lens = [max(L, 1) for L in lens]
    begin = [1]
    for n in new:
        begin.append(begin[-1] + n)
    N = begin[-1] + 3
    if falls:  # everything from one entry on begins again lower down
        at = B - B // 4
        down = begin[at] // 2
        begin = begin[:at] + [x - down for x in begin[at:]]
    walk(begin, lens, N, 3, G, 1, 64, 16, dtype, bits, 103)


def test_a_window_as_long_as_any_is_no_window():
    """The list of a cache beyond L2 is cut the same way, so the bits are the same."""
    L, n = 40000, 2048
    g = gen(104)
    pool, table = make_pool(g, [L], 64, 16, 8, 128, BF, 0)
    batch = api.PoolBatch(table, torch.tensor([L], device="cuda"), torch.tensor([0, n], device="cuda"), tokens=n, max_new=n)
    q = randn(g, n, 16, 128, dtype=BF)
    want = lod.lod_pool_attend(pool, batch, q)
    for window in (L, 1 << 40, (1 << 63) - n, (1 << 63) - 1):
        assert torch.equal(lod.lod_pool_attend(pool, batch, q, window=window), want), window


def test_outputs_whose_rows_overlap_are_refused():
    g = gen(105)
    pool, table = make_pool(g, [50, 60], 16, 4, 2, 64, BF, 0)
    batch = api.PoolBatch(table, torch.tensor([50, 60], device="cuda"), torch.tensor([0, 2, 5], device="cuda"), tokens=5,
                          max_new=3)
    q, k = randn(g, 5, 4, 64, dtype=BF), randn(g, 5, 2, 64, dtype=BF)
    one = torch.zeros(1, 4, 64, dtype=BF, device="cuda")
    for bad in (one.expand(5, 4, 64), torch.zeros(5, 1, 64, dtype=BF, device="cuda").expand(5, 4, 64)):
        with pytest.raises(lod.LodError, match="overlap"):
            lod.lod_pool_attend(pool, batch, q, out=bad)
        with pytest.raises(lod.LodError, match="overlap"):
            lod.lod_pool_append(pool, batch, k, k, rope=api.Rope(), q=q, q_out=bad)
    row = torch.zeros(1, 2, 64, 64, dtype=BF, device="cuda").expand(2, 2, 64, 64)
    with pytest.raises(lod.LodError, match="overlap"):
        lod.lod_pool_read(pool, batch, row, row)
    p = lod.Params(B=2, Hq=4, Hkv=2, d=64, Tmax=256, dtype=BF)
    cache = torch.zeros(1, 2, 256, 64, dtype=BF, device="cuda").expand(2, 2, 256, 64)
    k1 = randn(g, 2, 2, 3, 64, dtype=BF)
    with pytest.raises(lod.LodError, match="overlap"):
        lod.lod_append_rope(p, api.Rope(), None, k1, k1, cache, cache, torch.tensor([9, 9], device="cuda"))


# ------------------------------------------------------------------ long prompts of fp32

@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("Hq, Hkv, d, block, rot, inter", [(6, 2, 128, 64, 64, False), (4, 1, 64, 16, 64, True),
                                                           (8, 8, 128, 128, 24, False)])
def test_long_fp32_prompts(Hq, Hkv, d, block, rot, inter, bits):
    """Appends of thousands of fp32 tokens: more than the GPU holds warps for, into fp32 and 8-bit rows."""
    g = gen(106)
    lens, new = [6100, 3000, 5], [5000, 2999, 0]
    pool, table = make_pool(g, lens, block, Hq, Hkv, d, F32, bits)
    begin = [0, 5000, 7999, 7999]
    batch = api.PoolBatch(table, torch.tensor(lens, device="cuda"), torch.tensor(begin, device="cuda"), tokens=7999,
                          max_new=5000)
    rope, w = make_rope(g, d, F32, rot, inter, True)
    q, k, v = randn(g, 7999, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lod.lod_pool_append(pool, batch, k, v, rope=rope, q=q, status=status)
    assert int(status) == 0
    for b in range(2):
        L, n = lens[b], new[b]
        rows, pos = slice(begin[b], begin[b + 1]), torch.arange(L - n, L, device="cuda")
        y, mag = pt.rotate64(q[rows].transpose(0, 1), w[0], pos, rope.inv_freq, inter, 1e-5)
        close(out[rows].transpose(0, 1), y, rope_tol(y, mag, F32), "q")
        y, mag = (x.transpose(0, 1) for x in pt.rotate64(k[rows].transpose(0, 1), w[1], pos, rope.inv_freq, inter, 1e-5))
        rk, rv = pt.pool_rows(pool, table[b], pos)
        if bits:  # (as the small prompts: nearest codes of values within 2^-19 of the pair's size)
            e = pt.exponent64(y.float()).double()
            close(rk, y, 2.0 ** -4 * y.abs() + torch.exp2(e - 9)[..., None] + 2.0 ** -18 * mag, "K")
            c, ev = pt.quantise64(v[rows])
            assert torch.equal(rv, pt.codes_to_float(c) * torch.exp2(ev.double() - 127)[..., None])
        else:
            close(rk, y, rope_tol(y, mag, F32), "K")
            assert torch.equal(rv, v[rows].double())
