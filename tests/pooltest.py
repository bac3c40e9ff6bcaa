"""Plain 64-bit forms of the projections' append, the block pool's format and its attention, and the error bounds
that the kernels' arithmetic allows.

Bounds.  A value computed in fp32 and rounded once to type T is off by at most eps(T)/2 of itself plus the fp32 error
of its computation:
  * norm and rotation: mean of d <= 128 squares (fp32 sum by halves: at most 11 roundings), square root, two products
    and a sum of two products, an angle off by pi * 2^-24 and a sine and cosine off by 2 ulp: together below
    32 * 2^-24 = 2^-19 of |y1| + |y2| of the channel's pair;
  * a score: d products and sums, at most d * 2^-24 of sum |q_i k_i|, times the scale; a softmax weight is off by
    twice the largest score error of its row (numerator and denominator), plus 2^-20 for the exponentials and the
    scaling by log2 e (scores up to 2^4);
  * an output channel: sum_j p_j |v_j| times the weights' error, plus the sum's own roundings (a key tile's sums are
    joined in fp32: at most length * 2^-24), plus, in bf16, 2^-8 for weights rounded to bf16.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rotate64(x, w, pos, freq, interleaved, eps):
    """Rows x [..., tokens, d] at positions pos [tokens]: normed (w not None) and rotated, fp64.  Also the magnitude
    |y1| + |y2| of each channel's pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs()
    rot = 0 if freq is None else 2 * freq.numel()
    if rot:
        a = pos.double()[:, None] * freq.double()[None]
        i = torch.arange(rot // 2, device=x.device)
        i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y1, y2 = x[..., i1], x[..., i2]
        y[..., i1] = y1 * torch.cos(a) - y2 * torch.sin(a)
        y[..., i2] = y2 * torch.cos(a) + y1 * torch.sin(a)
        mag[..., i1] = mag[..., i2] = y1.abs() + y2.abs()
    return y, mag


def exponent64(x):
    """Row exponents e: the least with max|x| <= 448 * 2^e, clamped to [-120, 119]; found by counting up."""
    a = x.double().abs().amax(-1)
    e = torch.full(a.shape, -120, dtype=torch.int64, device=x.device)
    for k in range(-120, 119):
        e += a > 448.0 * 2.0 ** k
    return e


def quantise64(x):
    """(code bytes, exponent bytes) of finite rows x by comparison with every e4m3 value: nearest, ties to even."""
    e = exponent64(x)
    r = (x.double() * torch.exp2(-e.double())[..., None]).clamp(-448, 448)
    codes = torch.arange(127, dtype=torch.uint8, device=x.device)  # 0 .. 0x7e: the non-negative values in order
    vals = codes_to_float(codes)
    m = r.abs()
    hi = torch.searchsorted(vals, m).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = m - vals[lo], vals[hi] - m
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).to(torch.uint8)
    pick = torch.where(torch.signbit(x), pick | 0x80, pick)
    return pick, (e + 127).to(torch.uint8)


def codes_to_float(c):
    """e4m3 values of code bytes, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = c.to(torch.int64)
    ex, man = (c >> 3) & 15, (c & 7).double()
    v = torch.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * torch.exp2(ex.double() - 7))
    return torch.where(c >= 128, -v, v)


def pool_rows(pool, table_row, t):
    """fp64 rows [len(t), Hkv, d] of tokens t (K and V) of one sequence."""
    blk, off = table_row.long()[t // pool.block], t % pool.block
    out = []
    for X, E in ((pool.K, pool.Ke), (pool.V, pool.Ve)):
        if pool.bits:
            c = X.view(torch.uint8)[blk, :, off]
            out.append(codes_to_float(c) * torch.exp2(E[blk, :, off].double() - 127)[..., None])
        else:
            out.append(X[blk, :, off].double())
    return out


def attend64(pool, table, lens, begin, q, window=0, scale=None, bad_keys=None):
    """fp64 outputs and lse of every packed row, and their error bounds; rows no sequence owns are NaN.
    bad_keys: per sequence, a truth value per key that is left out."""
    N, Hq, d = q.shape
    G = Hq // pool.Hkv
    scale = scale or 1 / math.sqrt(d)
    dev = q.device
    o = torch.full((N, Hq, d), math.nan, dtype=torch.float64, device=dev)
    z = torch.full((N, Hq), math.nan, dtype=torch.float64, device=dev)
    to, tz = torch.zeros_like(o), torch.zeros_like(z)
    half = HALF[pool.dtype]
    for b in range(len(lens)):
        r0, r1, L = begin[b], begin[b + 1], lens[b]
        if r1 == r0:
            continue
        K, V = pool_rows(pool, table[b], torch.arange(L, device=dev))
        pos = torch.arange(L - (r1 - r0), L, device=dev)
        key = torch.arange(L, device=dev)
        seen = key[None] <= pos[:, None]
        if window:
            seen &= key[None] > pos[:, None] - window
        if bad_keys is not None:
            seen &= ~bad_keys[b][None]
            V = torch.where(bad_keys[b][:, None, None], torch.zeros_like(V), V)
            K = torch.where(bad_keys[b][:, None, None], torch.zeros_like(K), K)
        for h in range(Hq):
            k, v, x = K[:, h // G], V[:, h // G], q[r0:r1, h].double()
            s = (x @ k.t() * scale).masked_fill(~seen, -math.inf)
            mag = (x.abs() @ k.abs().t() * abs(scale)).masked_fill(~seen, 0).amax(-1)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
            z[r0:r1, h] = lse
            fin = torch.isfinite(v)
            v = torch.where(fin, v, torch.zeros_like(v))
            o[r0:r1, h] = p @ v
            o[r0:r1, h] += torch.where(seen.double() @ (~fin).double() > 0, math.nan, 0.0)  # (0 * NaN is NaN: only what is seen)
            spread = p @ v.abs()
            ds = (d + 2) * 2.0 ** -24 * mag
            tz[r0:r1, h] = ds + 2.0 ** -20 + L * 2.0 ** -24 + 2.0 ** -23 * lse.abs().nan_to_num(0, 0, 0)
            rel = 2 * ds + 2.0 ** -20 + L * 2.0 ** -24 + (2.0 ** -8 if pool.dtype == torch.bfloat16 else 0)
            to[r0:r1, h] = rel[:, None] * spread + half * o[r0:r1, h].abs() + 2.0 ** -120
    return o, z, to, tz
