"""The projections' append, the block pool's format and its attention on the GPU, against the 64-bit forms and the
derived bounds of tests/pooltest.py."""
import math

import pytest
import torch

import hierarchical_long_context_b200 as lod
from hierarchical_long_context_b200 import _lib, api
from tests import pooltest as pt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ST = dict(seqlen=1, page=2)


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def freqs(rot):
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    return (1e6 ** (-2.0 * i / rot)).float()


def close(got, want, tol, what):
    got = got.double()
    both = torch.isnan(got) & torch.isnan(want) | (got == want)
    off = torch.where(both, torch.zeros_like(want), (got - want).abs() - tol)
    bad = ~(off <= 0)
    assert not bad.any(), "%s: %d of %d outside, first at %s: got %r want %r bound %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(),
        tol.expand_as(want)[bad][0].item())


def make_rope(g, d, dtype, rot, inter, norm):
    w = [(1 + 0.3 * randn(g, d)).to(dtype) if norm else None for _ in range(2)]
    return api.Rope(freqs(rot) if rot else None, q_norm=w[0], k_norm=w[1], interleaved=inter, eps=1e-5), w


def rope_tol(y, mag, dtype):
    return pt.HALF[dtype] * y.abs() + 2.0 ** -19 * mag


# ------------------------------------------------------------------ dense append

@pytest.mark.parametrize("B, Hq, Hkv, d, n, dtype, rot, inter, norm", [
    (1, 1, 1, 64, 1, F32, 64, False, False),
    (3, 8, 8, 128, 1, BF, 128, False, True),
    (2, 8, 2, 128, 37, BF, 128, True, True),
    (2, 8, 1, 64, 5, BF, 32, False, True),
    (1, 4, 4, 128, 9, F32, 24, False, True),     # a pair distance that no 16-byte piece divides
    (2, 2, 2, 64, 3, BF, 24, False, False),
    (1, 8, 2, 64, 130, F32, 40, True, True),
    (1, 3, 3, 128, 2, BF, 0, False, True),       # norm alone
    (1, 16, 2, 128, 2500, BF, 128, False, True),
])
def test_dense_append(B, Hq, Hkv, d, n, dtype, rot, inter, norm):
    g = gen(1)
    Tmax = 4096
    p = lod.Params(B=B, Hq=Hq, Hkv=Hkv, d=d, Tmax=Tmax, dtype=dtype)
    rope, w = make_rope(g, d, dtype, rot, inter, norm)
    fused = randn(g, B, n, Hq + 2 * Hkv, d, dtype=dtype)
    q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], 2))
    lens = torch.tensor([n + 11 * b + (Tmax - n - 50 if b == 0 else 0) for b in range(B)], device="cuda")
    K = randn(g, B, Hkv, Tmax, d, dtype=dtype)
    V = randn(g, B, Hkv, Tmax, d, dtype=dtype)
    wantK, wantV = K.double(), V.double()
    tolK = torch.zeros_like(wantK)
    out = lod.lod_append_rope(p, rope, q, k, v, K, V, lens)
    assert out.shape == (B, Hq, n, d) and out.is_contiguous()
    for b in range(B):
        pos = torch.arange(int(lens[b]) - n, int(lens[b]), device="cuda")
        y, mag = pt.rotate64(q[b], w[0], pos, rope.inv_freq, inter, 1e-5)
        close(out[b], y, rope_tol(y, mag, dtype), "q %d" % b)
        y, mag = pt.rotate64(k[b], w[1], pos, rope.inv_freq, inter, 1e-5)
        wantK[b, :, pos], tolK[b, :, pos] = y, rope_tol(y, mag, dtype)
        wantV[b, :, pos] = v[b].double()
    close(K, wantK, tolK, "K")  # rows outside the new positions: unchanged
    assert torch.equal(V.double(), wantV)
    # keys and values alone, and queries in place
    K2 = K.clone()
    lod.lod_append_rope(p, rope, None, k, v, K2, V, lens)
    assert torch.equal(K2, K)
    q2 = q.clone(memory_format=torch.preserve_format)
    assert lod.lod_append_rope(p, rope, q2, k, v, K2, V, lens, q_out=q2) is q2
    assert torch.equal(q2, out)


def test_dense_append_far_positions():
    """At position 2^20 the angle of the first pair is 2^20 radian: a product in fp32 would be off by 2^-4."""
    g = gen(2)
    Tmax = 1 << 20
    p = lod.Params(B=1, Hq=2, Hkv=1, d=64, Tmax=Tmax, dtype=F32)
    rope, w = make_rope(g, 64, F32, 64, False, True)
    q, k = randn(g, 1, 2, 3, 64), randn(g, 1, 1, 3, 64)
    K = torch.zeros(1, 1, Tmax, 64, device="cuda")
    out = lod.lod_append_rope(p, rope, q, k, k, K, torch.zeros_like(K), torch.tensor([Tmax], device="cuda"))
    pos = torch.arange(Tmax - 3, Tmax, device="cuda")
    y, mag = pt.rotate64(q[0], w[0], pos, rope.inv_freq, False, 1e-5)
    close(out[0], y, rope_tol(y, mag, F32), "q")


def test_dense_append_skips_bad_lengths():
    g = gen(3)
    p = lod.Params(B=4, Hq=2, Hkv=1, d=64, Tmax=256, dtype=BF)
    rope, _ = make_rope(g, 64, BF, 64, False, False)
    K = randn(g, 4, 1, 256, 64, dtype=BF)
    V, K0 = K.clone(), K.clone()
    q, k = randn(g, 4, 2, 2, 64, dtype=BF), randn(g, 4, 1, 2, 64, dtype=BF)
    out = torch.full_like(q, 7.0)
    lens = torch.tensor([1, 257, -5, 2], device="cuda")
    lod.lod_append_rope(p, rope, q, k, k, K, V, lens, q_out=out)
    assert torch.equal(K[:3], K0[:3]) and (out[:3] == 7).all()
    assert torch.equal(V[3, :, :2], k[3]) and torch.equal(V[3, :, 2:], K0[3, :, 2:])


# ------------------------------------------------------------------ pool set-up

def make_pool(g, lens, block, Hq, Hkv, d, dtype, bits, slack=2, fill="random"):
    """A pool whose blocks are dealt out at random; unused rows and blocks hold NaN (or random codes)."""
    need = [-(-L // block) for L in lens]
    width = max(max(need), 1) + 1
    blocks = sum(need) + slack
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    pool = api.Pool.empty(blocks, block, Hq, Hkv, d, dtype, bits)
    for X, E in ((pool.K, pool.Ke), (pool.V, pool.Ve)):
        if bits:
            X.fill_(0x7f)
            E.fill_(255)
        else:
            X.fill_(math.nan)
    for b, L in enumerate(lens):
        t = torch.arange(L, device="cuda")
        blk, off = table[b].long()[t // block], t % block
        for X, E, s in ((pool.K, pool.Ke, 1.0), (pool.V, pool.Ve, 1.0)):
            x = (randn(g, L, Hkv, d) * s).to(dtype)
            if bits and L:
                c, e = pt.quantise64(x)
                X[blk, :, off], E[blk, :, off] = c, e
            else:
                X[blk, :, off] = x
    return pool, table


def make_batch(table, lens, new, gap=0):
    """new tokens packed with `gap` unowned rows before the first and behind the last."""
    begin = [gap]
    for n in new:
        begin.append(begin[-1] + n)
    return begin, api.PoolBatch(table, torch.tensor(lens, device="cuda"), torch.tensor(begin, device="cuda"),
                                tokens=begin[-1] + gap, max_new=max(max(new), 1))


# ------------------------------------------------------------------ pool append and read

@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("Hq, Hkv, d, block, dtype, rot, inter, norm", [
    (8, 2, 128, 16, BF, 128, False, True),
    (4, 4, 64, 32, BF, 24, True, False),
    (6, 2, 128, 64, F32, 64, False, True),
    (1, 1, 64, 128, F32, 40, False, True),
])
def test_pool_append_and_read(Hq, Hkv, d, block, dtype, rot, inter, norm, bits):
    g = gen(5)
    lens, new = [1, 300, 17, 64, 129], [1, 300, 3, 0, 20]
    pool, table = make_pool(g, lens, block, Hq, Hkv, d, dtype, bits)
    begin, batch = make_batch(table, lens, new, gap=2)
    N = batch.tokens
    rope, w = make_rope(g, d, dtype, rot, inter, norm)
    fused = randn(g, N, Hq + 2 * Hkv, d)
    fused[:, :, ::16] *= 8
    q, k, v = fused.to(dtype).split([Hq, Hkv, Hkv], 1)
    before = [pt.pool_rows(pool, table[b], torch.arange(L, device="cuda")) for b, L in enumerate(lens)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((N, Hq, d), 5.0, dtype=dtype, device="cuda")
    lod.lod_pool_append(pool, batch, k, v, rope=rope, q=q, q_out=out, status=status)
    assert (out[:2] == 5).all() and (out[-2:] == 5).all()
    T = 512
    Kd = torch.full((len(lens), Hkv, T, d), 3.0, dtype=dtype, device="cuda")
    Vd = Kd.clone()
    lod.lod_pool_read(pool, batch, Kd, Vd, status=status, t_end=block * table.shape[1] if block * table.shape[1] < T else T)
    assert int(status) == 0
    for b, L in enumerate(lens):
        n = new[b]
        pos = torch.arange(L - n, L, device="cuda")
        rows = slice(begin[b], begin[b + 1])
        if n:
            y, mag = pt.rotate64(q[rows].transpose(0, 1), w[0], pos, rope.inv_freq, inter, 1e-5)
            close(out[rows].transpose(0, 1), y, rope_tol(y, mag, dtype), "q")
        rk, rv = pt.pool_rows(pool, table[b], torch.arange(L, device="cuda"))
        y, mag = pt.rotate64(k[rows].transpose(0, 1), w[1], pos, rope.inv_freq, inter, 1e-5)
        y, mag, x = y.transpose(0, 1), mag.transpose(0, 1), v[rows]
        if bits:
            # nearest code of a value within 2^-19 mag of y; the exponent may go by a maximum that far off
            e = pt.exponent64(y.float()).double() if n else torch.zeros(0, Hkv, device="cuda")
            tol = 2.0 ** -4 * y.abs() + torch.exp2(e - 9)[..., None] + 2.0 ** -18 * mag
            close(rk[L - n:], y, tol, "K")
            c, ev = pt.quantise64(x)
            assert torch.equal(rv[L - n:], pt.codes_to_float(c) * torch.exp2(ev.double() - 127)[..., None])
        else:
            close(rk[L - n:], y, rope_tol(y, mag, dtype), "K")
            assert torch.equal(rv[L - n:], x.double())
        assert torch.equal(rk[: L - n], before[b][0][: L - n]) and torch.equal(rv[: L - n], before[b][1][: L - n])
        # the read-back is exact (a code times a power of two fits bf16), and leaves other rows alone
        assert torch.equal(Kd[b, :, :L].double(), rk.transpose(0, 1)) and torch.equal(Vd[b, :, :L].double(), rv.transpose(0, 1))
        assert (Kd[b, :, L:] == 3).all() and (Vd[b, :, L:] == 3).all()
    # a range of the tokens, into a strided cache
    wide = torch.full((len(lens), T, Hkv, 2 * d), 4.0, dtype=dtype, device="cuda")
    Ks, Vs = (wide[..., i * d:(i + 1) * d].transpose(1, 2) for i in range(2))
    lod.lod_pool_read(pool, batch, Ks, Vs, 60, 131)
    for b, L in enumerate(lens):
        hi = min(L, 131)
        if hi > 60:
            assert torch.equal(Ks[b, :, 60:hi], Kd[b, :, 60:hi]) and torch.equal(Vs[b, :, 60:hi], Vd[b, :, 60:hi])
        assert (wide[b, :60] == 4).all() and (wide[b, max(hi, 60):] == 4).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantised_rows_are_the_nearest_codes(dtype):
    """Rows without rope, so the stored bytes are fixed: borders between codes, ties, subnormal codes, rows of zeros,
    tiny and huge rows, and rows that hold infinities or NaN."""
    g = gen(6)
    d, rows = 64, 96
    x = randn(g, rows, 2, d) * torch.exp2(torch.randint(-30, 30, (rows, 2, 1), generator=g, device="cuda").float())
    x[0] = 0
    x[1, 0] = 448.0
    x[1, 1] = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item() if dtype == F32 else 450.0
    c = pt.codes_to_float(torch.arange(127, dtype=torch.uint8, device="cuda")).float()
    mid = (c[1:] + c[:-1]) / 2  # ties
    x[2, 0], x[2, 1] = mid[:64], -mid[62:126]
    x[2, :, 0] = 448.0
    x[3] = 2.0 ** -125
    x[4, 0], x[4, 1] = 3e38, -1.7e38
    x[5, 0] = randn(g, d) * 2.0 ** -128
    x[6, 0, 3] = 448 * 2.0 ** 20
    x = x.to(dtype)
    want_c, want_e = pt.quantise64(x)
    x[7, 0, 5], x[7, 1, 6], x[8, 0, 0] = math.inf, math.nan, -math.inf
    lens = [rows]
    pool, table = make_pool(g, lens, 32, 2, 2, d, dtype, 8)
    _, batch = make_batch(table, lens, [rows])
    lod.lod_pool_append(pool, batch, x, x)
    t = torch.arange(rows, device="cuda")
    blk, off = table[0].long()[t // 32], t % 32
    codes, e = pool.K[blk, :, off], pool.Ke[blk, :, off]
    special = ~torch.isfinite(x.float()).all(-1)
    assert special.sum() == 3
    assert (e[special] == 255).all() and (codes[special] == 0x7f).all()
    assert torch.equal(e[~special], want_e[~special])
    got, want = codes[~special], want_c[~special]
    assert torch.equal(pt.codes_to_float(got), pt.codes_to_float(want))
    assert torch.equal(pool.V[blk, :, off], codes) and torch.equal(pool.Ve[blk, :, off], e)
    Kd = torch.zeros(1, 2, 96, d, dtype=dtype, device="cuda")
    Vd = torch.zeros_like(Kd)
    lod.lod_pool_read(pool, batch, Kd, Vd)
    back = Kd[0].transpose(0, 1)
    assert torch.isnan(back[special]).all() and torch.isfinite(back[~special]).all()


def test_bad_blocks_and_refused_sequences_are_reported():
    g = gen(7)
    lens, new = [40, 40, 40, 200, 30], [2, 2, 2, 2, 2]
    pool, table = make_pool(g, [40, 40, 40, 40, 30], 16, 4, 2, 64, BF, 0)
    table[1, 2] = pool.K.shape[0]          # the newest tokens' block
    table[2, 0] = -7                       # an old block
    begin, batch = make_batch(table, lens, new)  # sequence 3 is longer than its table row
    ref = pool.K.clone()
    k = randn(g, 10, 2, 64, dtype=BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lod.lod_pool_append(pool, batch, k, k, status=status)
    assert int(status) == ST["seqlen"] | ST["page"]
    for b in (0, 2, 4):
        t = torch.arange(lens[b] - 2, lens[b], device="cuda")
        assert torch.equal(pool.K[table[b].long()[t // 16], :, t % 16], k[2 * b:2 * b + 2])
    changed = (pool.K.view(torch.int16) != ref.view(torch.int16)).any(-1).any(1).sum()
    assert int(changed) == 6
    status.zero_()
    Kd = torch.full((5, 2, 48, 64), 3.0, dtype=BF, device="cuda")
    Vd = Kd.clone()
    lod.lod_pool_read(pool, batch, Kd, Vd, status=status)
    assert int(status) == ST["seqlen"] | ST["page"]
    assert (Kd[3] == 3).all() and (Kd[2, :, :16] == 3).all() and (Kd[1, :, 32:] == 3).all()
    assert (Kd[2, :, 16:40] != 3).any() and (Kd[0, :, 40:] == 3).all()


# ------------------------------------------------------------------ attention

def run_attend(pool, table, lens, new, seed, window=0, scale=0.0, qmul=1.0, gap=0):
    g = gen(seed)
    begin, batch = make_batch(table, lens, new, gap)
    N, Hq, d, dt = batch.tokens, pool.Hq, pool.d, pool.dtype
    q = (randn(g, N, Hq, d) * qmul).to(dt)
    out = torch.full((N, Hq, d), 9.0, dtype=dt, device="cuda")
    lse = torch.full((N, Hq), 9.0, device="cuda")
    ws = api.pool_workspace(pool, batch)
    lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, window=window, scale=scale, ws=ws)
    return begin, batch, q, out, lse, ws


def check_attend(pool, table, lens, new, seed, window=0, scale=0.0, qmul=1.0, gap=0):
    begin, batch, q, out, lse, ws = run_attend(pool, table, lens, new, seed, window, scale, qmul, gap)
    o, z, to, tz = pt.attend64(pool, table, lens, begin, q, window, scale)
    own = torch.zeros(batch.tokens, dtype=torch.bool, device="cuda")
    own[begin[0]:begin[-1]] = True
    assert lod.lod_get_status(ws) == 0
    close(lse[own], z[own], tz[own], "lse")
    close(out[own], o[own], to[own], "out")
    assert (out[~own] == 9).all() and (lse[~own] == 9).all()
    return q, out, lse


SHAPES = [  # Hq, Hkv, d, block, lens, new, window
    (1, 1, 64, 16, [1], [1], 0),
    (1, 1, 64, 16, [4096], [1], 0),
    (8, 1, 128, 16, [257], [1], 0),
    (8, 8, 128, 64, [1000, 31, 128, 129], [1, 1, 1, 1], 0),
    (64, 8, 128, 64, [3000, 5, 700], [1, 1, 1], 0),
    (16, 8, 64, 32, [640, 1], [1, 1], 100),
    (12, 4, 128, 128, [513, 512, 511], [2, 5, 1], 0),       # G = 3
    (10, 2, 64, 16, [100, 2000], [3, 7], 33),               # G = 5
    (16, 1, 128, 32, [900], [4], 0),                        # 64 rows
    (16, 1, 128, 32, [900], [5], 0),                        # 80 rows
    (64, 1, 64, 32, [300, 77], [2, 1], 0),                  # G = 64
    (8, 2, 128, 16, [77, 77], [77, 77], 0),                 # whole prompts
    (4, 4, 128, 64, [1500], [700], 0),
    (4, 1, 128, 64, [2100], [300], 256),
    (6, 2, 64, 64, [600, 1300, 40, 9], [450, 1, 40, 0], 0), # mixed, one without new tokens
    (2, 2, 128, 128, [1025, 385], [257, 129], 1),           # a window of the token itself
    (8, 8, 64, 16, [333] * 5, [111, 1, 64, 17, 128], 50),
    (32, 8, 128, 32, [2049], [1024], 0),
]


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0), (F32, 8)])
@pytest.mark.parametrize("Hq, Hkv, d, block, lens, new, window", SHAPES)
def test_attend(Hq, Hkv, d, block, lens, new, window, dtype, bits):
    pool, table = make_pool(gen(11), lens, block, Hq, Hkv, d, dtype, bits)
    check_attend(pool, table, lens, new, 12, window=window)


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0)])
@pytest.mark.parametrize("n", [1, 40])
def test_attend_peaked_scores_and_gaps(n, dtype, bits):
    """Scores of +-60 and more: the running maximum moves by a lot; rows that no sequence owns around the batch."""
    lens = [900, 350]
    pool, table = make_pool(gen(13), lens, 32, 8, 2, 128, dtype, bits)
    check_attend(pool, table, lens, [n, n], 14, qmul=3.0, scale=0.7, gap=3)


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0)])
@pytest.mark.parametrize("n", [1, 100])
def test_attend_is_repeatable_and_follows_its_inputs(n, dtype, bits):
    lens = [5000, 1200, 130]
    pool, table = make_pool(gen(15), lens, 64, 16, 4, 128, dtype, bits)
    a = run_attend(pool, table, lens, [n, n, n], 16)
    b = run_attend(pool, table, lens, [n, n, n], 16)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])
    # other blocks for the same rows: the same bits
    perm = torch.randperm(pool.K.shape[0], generator=gen(17), device="cuda")
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm), device="cuda")
    pool2 = api.Pool(pool.K[perm], pool.V[perm], None if not bits else pool.Ke[perm], None if not bits else pool.Ve[perm],
                     Hq=16, dtype=dtype)
    t2 = torch.where(table >= 0, inv[table.clamp(min=0).long()].to(torch.int32), table)
    c = run_attend(pool2, t2.contiguous(), lens, [n, n, n], 16)
    assert torch.equal(a[3], c[3]) and torch.equal(a[4], c[4])


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0)])
@pytest.mark.parametrize("n", [1, 60])
def test_attend_bad_blocks_and_refused_sequences(n, dtype, bits):
    lens, new = [300, 300, 260, 100, 64], [n, n, n, n, n]
    pool, table = make_pool(gen(18), lens, 32, 4, 2, 64, dtype, bits)
    table[1, 1] = pool.K.shape[0] + 3      # keys 32 .. 63 of sequence 1 are left out
    table[4, :2] = -1                      # sequence 4 has no key at all
    bad = [torch.zeros(L, dtype=torch.bool, device="cuda") for L in lens]
    bad[1][32:64] = True
    bad[4][:] = True
    begin, batch = make_batch(table, lens, new)
    batch.seq_lens[3] = 1 << 40            # refused
    g = gen(19)
    q = randn(g, batch.tokens, 4, 64, dtype=dtype)
    lse = torch.full((batch.tokens, 4), 9.0, device="cuda")
    ws = api.pool_workspace(pool, batch)
    out = lod.lod_pool_attend(pool, batch, q, lse=lse, ws=ws)
    assert lod.lod_get_status(ws) == ST["seqlen"] | ST["page"]
    safe = table.clone()
    safe[1, 1] = 0
    safe[4, :2] = 0
    o, z, to, tz = pt.attend64(pool, safe, lens, begin, q, bad_keys=bad)
    r = slice(begin[3], begin[4])
    o[r], z[r], to[r], tz[r] = 0, -math.inf, 0, 0
    close(lse, z, tz, "lse")
    close(out, o, to, "out")
    assert (out[r] == 0).all() and (out[begin[4]:] == 0).all() and (lse[begin[4]:] == -math.inf).all()
    # prefix sums that fall, rows outside the call, too many new tokens, fewer tokens than new ones
    for wrong in ([0, n, 0, 3 * n, 4 * n, 5 * n], [0, n, 2 * n, 3 * n, 4 * n, 5 * n + 1], [-n, n, 2 * n, 3 * n, 4 * n, 5 * n]):
        batch.new_begin.copy_(torch.tensor(wrong, device="cuda"))
        lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, ws=ws)
        assert lod.lod_get_status(ws) & ST["seqlen"]
    batch.new_begin.copy_(torch.tensor(begin, device="cuda"))
    batch.seq_lens.copy_(torch.tensor([n - 1, 0, 0, -1, n], device="cuda"))
    lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, ws=ws)
    assert lod.lod_get_status(ws) & ST["seqlen"]
    assert (out == 0).all()


@pytest.mark.parametrize("n", [1, 90])
def test_attend_of_an_8_bit_pool_is_that_of_its_read_back(n):
    """A code times its power of two is exact in bf16, so both pools hold the same numbers."""
    lens = [777, 50 + n]
    pool, table = make_pool(gen(20), lens, 16, 8, 2, 128, BF, 8)
    _, batch = make_batch(table, lens, [n, n])
    T = 1024
    Kd = torch.zeros(2, 2, T, 128, dtype=BF, device="cuda")
    Vd = torch.zeros_like(Kd)
    lod.lod_pool_read(pool, batch, Kd, Vd, 0, min(T, table.shape[1] * 16))
    raw = api.Pool(*(x.unflatten(2, (T // 64, 64)).transpose(1, 2).reshape(-1, 2, 64, 128).contiguous() for x in (Kd, Vd)),
                   Hq=8, dtype=BF)
    t2 = torch.arange(2 * T // 64, dtype=torch.int32, device="cuda").view(2, -1)
    check_attend(pool, table, lens, [n, n], 21)
    q, out, lse = check_attend(raw, t2, lens, [n, n], 21)
    begin, batch, q8, out8, lse8, _ = run_attend(pool, table, lens, [n, n], 21)
    o, z, to, tz = pt.attend64(pool, table, lens, begin, q)
    close(out8, out.double(), 2 * to, "out")
    close(lse8, lse.double(), 2 * tz, "lse")


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 8)])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_attend_rows_of_many_sizes(n, dtype, bits):
    """Key and value rows of sizes 2^-8 to 2^6, queries 2^-10 and 2^10 at a matching scale, rows of zeros."""
    g = gen(50)
    lens = [700, 200]
    pool, table = make_pool(g, lens, 32, 8, 2, 128, dtype, 0)
    f = torch.exp2(torch.randint(-8, 7, (2, *pool.K.shape[:3], 1), generator=g, device="cuda").float())
    f[:, :, :, 3] = 0
    K, V = (pool.K.float().nan_to_num(0) * f[0].clamp(max=1)).to(dtype), (pool.V.float().nan_to_num(0) * f[1]).to(dtype)
    if bits:
        (kc, ke), (vc, ve) = pt.quantise64(K), pt.quantise64(V)
        pool = api.Pool(kc, vc, ke, ve, Hq=8, dtype=dtype)
    else:
        pool = api.Pool(K, V, Hq=8, dtype=dtype)
    for m in (2.0 ** -10, 1.0, 2.0 ** 10):
        check_attend(pool, table, lens, [n, n], 51, qmul=m, scale=0.1 / m)


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (BF, 8), (F32, 0), (F32, 8)])
@pytest.mark.parametrize("n", [1, 60])
def test_nan_and_infinite_rows_reach_only_the_queries_that_see_them(n, dtype, bits):
    """A sequence whose rows hold NaN and infinities, appended as such: its queries' outputs are NaN, the other
    sequence's, a window that ends before those rows, and keys behind the length are not touched."""
    g = gen(52)
    lens = [400, 333]
    pool, table = make_pool(g, lens, 16, 4, 2, 64, dtype, bits)
    begin, batch = make_batch(table, lens, [400, 0])
    k, v = randn(g, 400, 2, 64, dtype=dtype), randn(g, 400, 2, 64, dtype=dtype)
    k[5, :, 3], v[9, 0, 2] = math.nan, math.inf
    lod.lod_pool_append(pool, batch, k, v)
    begin, batch, q, out, lse, _ = run_attend(pool, table, lens, [n, n], 53)
    assert torch.isnan(out[:n].float()).all() and torch.isnan(lse[:n]).all()
    o, z, to, tz = pt.attend64(pool, table, lens, begin, q)
    close(out[n:], o[n:], to[n:], "out")
    close(lse[n:], z[n:], tz[n:], "lse")
    check_attend(pool, table, lens, [n, n], 54, window=250)


@pytest.mark.parametrize("dtype, bits", [(BF, 0), (F32, 8)])
def test_attend_strides_and_default_outputs(dtype, bits):
    lens, new = [200, 90], [1, 30]
    pool, table = make_pool(gen(22), lens, 16, 8, 2, 64, dtype, bits)
    begin, batch = make_batch(table, lens, new)
    wide = randn(gen(23), batch.tokens, 3 * 8 + 1, 64, dtype=dtype)
    q = wide[:, 1:25:3]
    out = lod.lod_pool_attend(pool, batch, q)
    assert torch.equal(out, lod.lod_pool_attend(pool, batch, q.contiguous()))
    o, _, to, _ = pt.attend64(pool, table, lens, begin, q)
    close(out, o, to, "out")
    buf = torch.zeros(batch.tokens, 8, 2, 64, dtype=dtype, device="cuda")
    lod.lod_pool_attend(pool, batch, q, out=buf[:, :, 1])
    assert torch.equal(buf[:, :, 1], out) and (buf[:, :, 0] == 0).all()
    # heads outermost
    t = torch.zeros(8, batch.tokens, 64, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(lod.lod_pool_attend(pool, batch, q.transpose(0, 1).contiguous().transpose(0, 1), out=t), out)


@pytest.mark.parametrize("dtype, bits, n", [(BF, 0, 1), (BF, 8, 1), (BF, 8, 50), (BF, 0, 50), (F32, 0, 20)])
def test_attend_captured_in_a_graph_follows_new_lengths(dtype, bits, n):
    """Lengths, tables and queries are read on the device: a captured call serves later steps."""
    lens = [700, 300]
    pool, table = make_pool(gen(24), lens, 32, 8, 2, 128, dtype, bits)
    begin, batch = make_batch(table, lens, [n, n])
    q = randn(gen(25), batch.tokens, 8, 128, dtype=dtype)
    out, lse = torch.zeros_like(q), torch.zeros(batch.tokens, 8, device="cuda")
    ws = api.pool_workspace(pool, batch)
    lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lod.lod_pool_attend(pool, batch, q, out=out, lse=lse, ws=ws)
    for lens2, swap in (([300, 300], False), ([555, 128], True), ([n, 299], False)):
        batch.seq_lens.copy_(torch.tensor(lens2, device="cuda"))
        if swap:
            q.copy_(randn(gen(26), *q.shape, dtype=dtype))
        graph.replay()
        o, z, to, tz = pt.attend64(pool, table, lens2, begin, q)
        close(out, o, to, "out")
        close(lse, z, tz, "lse")


def test_two_streams_with_workspaces_of_their_own():
    lens = [6000, 900]
    pool, table = make_pool(gen(27), lens, 64, 16, 2, 128, BF, 8)
    _, batch = make_batch(table, lens, [1, 1])
    qs = [randn(gen(28 + i), 2, 16, 128, dtype=BF) for i in range(2)]
    want = [lod.lod_pool_attend(pool, batch, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [api.pool_workspace(pool, batch) for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for i in range(20):
        for s in range(2):
            lod.lod_pool_attend(pool, batch, qs[s], out=outs[s][i], ws=ws[s], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(o, want[s]) for o in outs[s])


def test_small_workspaces_and_host_memory_are_refused():
    lens = [64]
    pool, table = make_pool(gen(30), lens, 16, 4, 2, 64, BF, 0)
    _, batch = make_batch(table, lens, [2])
    q = randn(gen(31), 2, 4, 64, dtype=BF)
    ws = api.pool_workspace(pool, batch)
    for bad in (ws[: ws.numel() - 256], torch.zeros(ws.numel() + 256, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(lod.LodError) as e:
            lod.lod_pool_attend(pool, batch, q, ws=bad)
        assert e.value.code == _lib.LOD_EINVAL
    with pytest.raises(lod.LodError) as e:
        lod.lod_pool_attend(pool, batch, q.cpu(), ws=ws)
    assert e.value.code == _lib.LOD_EINVAL
    # page-locked queries and outputs are used in place
    qh, oh = q.cpu().pin_memory(), torch.zeros(2, 4, 64, dtype=BF).pin_memory()
    lod.lod_pool_attend(pool, batch, qh, out=oh, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(oh.cuda(), lod.lod_pool_attend(pool, batch, q))


def test_long_sequence_offsets_pass_32_bits():
    """A pool of more than 2^32 bytes in K: the newest blocks sit behind the first 4 GB."""
    block, Hkv, d = 128, 8, 128
    blocks = (1 << 32) // (block * Hkv * d * 2) + 40
    pool = api.Pool.empty(blocks, block, 16, Hkv, d, BF, 0)
    g = gen(32)
    lens = [block * 30 - 7]
    table = torch.arange(blocks - 30, blocks, dtype=torch.int32, device="cuda")[None].contiguous()
    for X in (pool.K, pool.V):
        X[blocks - 30:] = randn(g, 30, Hkv, block, d, dtype=BF)
    check_attend(pool, table, lens, [1], 33)
    check_attend(pool, table, lens, [40], 34)
    begin, batch = make_batch(table, lens, [9])
    k = randn(g, 9, Hkv, d, dtype=BF)
    lod.lod_pool_append(pool, batch, k, k)
    Kd = torch.zeros(1, Hkv, lens[0], d, dtype=BF, device="cuda")
    Vd = torch.zeros_like(Kd)
    lod.lod_pool_read(pool, batch, Kd, Vd, lens[0] - 9, lens[0])
    assert torch.equal(Kd[0, :, -9:], k.transpose(0, 1)) and torch.equal(Vd, Kd)


@pytest.mark.parametrize("bits, window", [(0, 0), (8, 0), (0, 9000)])
def test_a_cache_beyond_l2_is_taken_in_rounds(bits, window):
    """164 MB of bf16 cache and more than 64 key tiles a CTA and round: the work list is walked in several rounds.
    Some heads against the 64-bit form, all of them against calls of fewer rows."""
    L, n = 40000, 2048
    pool, table = make_pool(gen(60), [L], 64, 16, 8, 128, BF, bits)
    begin, batch, q, out, lse, ws = run_attend(pool, table, [L], [n], 61, window=window)
    assert lod.lod_get_status(ws) == 0
    for h in (0, 7):  # KV heads, as pools of one head
        cut = [None if x is None else x[:, h:h + 1].contiguous() for x in (pool.K, pool.V, pool.Ke, pool.Ve)]
        one = api.Pool(*cut, Hq=2, dtype=BF)
        for lo in (0, n - 40):
            Lr = L - n + lo + 40
            o, z, to, tz = pt.attend64(one, table, [Lr], [0, 40], q[lo:lo + 40, 2 * h:2 * h + 2], window)
            close(out[lo:lo + 40, 2 * h:2 * h + 2], o, to, "out")
            close(lse[lo:lo + 40, 2 * h:2 * h + 2], z, tz, "lse")
    for lo, m in ((0, 100), (1000, 77)):  # another cut of the same rows: other partial sums, so bounds and not bits
        b2 = api.PoolBatch(table, torch.tensor([L - n + lo + m], device="cuda"), torch.tensor([0, m], device="cuda"),
                           tokens=m, max_new=m)
        z2 = torch.zeros(m, 16, device="cuda")
        o2 = lod.lod_pool_attend(pool, b2, q[lo:lo + m], lse=z2, window=window)
        # both within 2^-8 (weights) of sum p |v| <= max |v| < 6, and 2^-8 of themselves
        assert (o2.float() - out[lo:lo + m].float()).abs().max() < 2 * 6 * 2.0 ** -8
        assert (z2 - lse[lo:lo + m]).abs().max() < 1e-4


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("bits", [0, 8])
def test_prompt_and_decode_through_the_pool(bits):
    """A model's layer on the pool: a prompt in two chunks, then single tokens, each appended and attended, equals
    attention over all rows at once."""
    g = gen(40)
    Hq, Hkv, d, block, total = 8, 2, 128, 32, 330
    rope, w = make_rope(g, d, BF, 128, False, True)
    pool = api.Pool.empty(24, block, Hq, Hkv, d, BF, bits)
    table = torch.randperm(24, generator=g, device="cuda").to(torch.int32).view(2, 12)
    x = randn(g, 2, total, Hq + 2 * Hkv, d, dtype=BF)
    got = torch.zeros(2, total, Hq, d, dtype=BF, device="cuda")
    qrot = torch.zeros_like(got)
    at = 0
    for n in (200, 127, 1, 1, 1):
        fused = x[:, at:at + n].reshape(2 * n, Hq + 2 * Hkv, d)
        q, k, v = fused.split([Hq, Hkv, Hkv], 1)
        at += n
        batch = api.PoolBatch(table, torch.tensor([at, at], device="cuda"), torch.tensor([0, n, 2 * n], device="cuda"),
                              tokens=2 * n, max_new=n)
        qr = lod.lod_pool_append(pool, batch, k, v, rope=rope, q=q)
        qrot[:, at - n:at] = qr.view(2, n, Hq, d)
        got[:, at - n:at] = lod.lod_pool_attend(pool, batch, qr).view(2, n, Hq, d)
    begin = [0, total, 2 * total]
    o, _, to, _ = pt.attend64(pool, table, [total, total], begin, qrot.view(2 * total, Hq, d))
    close(got.view(2 * total, Hq, d), o, to, "out")


def test_pool_feeds_the_lod_path():
    """A sequence kept in the 8-bit pool is read back into the dense cache, indexed, extended with lod_append_rope and
    decoded: with a window over everything the LoD decode is exact attention, and equals the pool's."""
    g = gen(41)
    Hq, Hkv, d, T, block = 8, 2, 128, 1024, 64
    rope, w = make_rope(g, d, BF, 128, False, True)
    pool = api.Pool.empty(20, block, Hq, Hkv, d, BF, 8)
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None].contiguous()
    n = 700
    batch = api.PoolBatch(table, torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda"), tokens=n, max_new=n)
    k, v = randn(g, n, Hkv, d, dtype=BF), randn(g, n, Hkv, d, dtype=BF)
    lod.lod_pool_append(pool, batch, k, v, rope=rope)
    p = lod.Params(B=1, Hq=Hq, Hkv=Hkv, d=d, Tmax=T, dtype=BF, window=1024)
    K = torch.zeros(1, Hkv, T, d, dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    lod.lod_pool_read(pool, batch, K, V)
    ix = lod.Index(p)
    lod.lod_build_index(p, K, V, 0, n // 256, ix)
    lens = torch.tensor([n + 1], device="cuda")
    q, k1, v1 = randn(g, 1, Hq, 1, d, dtype=BF), randn(g, 1, Hkv, 1, d, dtype=BF), randn(g, 1, Hkv, 1, d, dtype=BF)
    qr = lod.lod_append_rope(p, rope, q, k1, v1, K, V, lens)
    out = lod.lod_decode(p, qr.view(1, Hq, d), K, V, lens, ix)
    # the same in exact attention over a pool that holds the dense cache's rows
    raw = api.Pool(*(x[0].unflatten(1, (16, 64)).transpose(0, 1).contiguous() for x in (K, V)), Hq=Hq, dtype=BF)
    one = api.PoolBatch(table, lens, torch.tensor([0, 1], device="cuda"), tokens=1, max_new=1)
    got = lod.lod_pool_attend(raw, one, qr.view(1, Hq, d))
    o, _, to, _ = pt.attend64(raw, table, [n + 1], [0, 1], qr.view(1, Hq, d))
    close(got, o, to, "pool")
    close(out, o, to + 2.0 ** -8 * o.abs(), "lod")
