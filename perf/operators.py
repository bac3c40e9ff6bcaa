"""Cases, plain forms and exact values of the cache operators: norm + rotation + append, the block pool's
quantised write and read-back, and the attention of new tokens over the block pool.

`listed()` gives the cases, `draw(rng)` another of the same ranges, `prepare(case, seed)` a case's inputs,
`run(state)` one pass (the plain form in torch, or this repository's kernels where `own` is true), `exact(case, seed)`
the values from the definitions in 64 bits, and `work(case)` the bytes and operations a pass cannot do without.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_THETA = 1e6
_EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of the single-head fp32 model: the smallest call, where latency is all there is
        dict(name="append_tiny_f32", op="append", B=1, n=1, len=4096, Tmax=4096, Hq=1, Hkv=1, d=64, dtype="f32",
             rot=64, interleaved=False, norm=False),
        # a decode step of eight sequences of a 64 / 8 head model
        dict(name="append_step_b8", op="append", B=8, n=1, len=4001, Tmax=4096, Hq=64, Hkv=8, d=128, dtype="bf16",
             rot=128, interleaved=False, norm=True),
        # a long prompt of a 32 / 8 head model written into the dense cache at once
        dict(name="append_prompt_32k", op="append", B=1, n=32768, len=32768, Tmax=32768, Hq=32, Hkv=8, d=128,
             dtype="bf16", rot=128, interleaved=False, norm=True),
        # a decode step into the 8-bit pool, and the 256-token chunk it completes read back for the index build
        dict(name="store_step_b8", op="store", B=8, n=1, len=4096, ragged=0, read=256, Hq=64, Hkv=8, d=128,
             dtype="bf16", block=16, bits=8, rot=128, interleaved=False, norm=True),
        # ragged prompts into the 8-bit pool, and every sequence read back into the dense cache
        dict(name="store_prompt_ragged", op="store", B=5, n=8000, len=32768, ragged=3, read=32768, Hq=32, Hkv=8, d=128,
             dtype="bf16", block=64, bits=8, rot=64, interleaved=True, norm=True),
        # fp32 rows kept as they are (no quantisation), odd lengths
        dict(name="store_raw_f32", op="store", B=3, n=333, len=4097, ragged=1, read=4097, Hq=8, Hkv=2, d=64,
             dtype="f32", block=32, bits=0, rot=32, interleaved=False, norm=True),
        # one token of the single-head fp32 model over 4096
        dict(name="attend_tiny_f32", op="attend", B=1, n=1, len=4096, ragged=0, Hq=1, Hkv=1, d=64, dtype="f32",
             block=16, bits=0, window=0),
        # a decode step at 32K, batch 8
        dict(name="attend_step_32k_b8", op="attend", B=8, n=1, len=32768, ragged=0, Hq=64, Hkv=8, d=128, dtype="bf16",
             block=64, bits=0, window=0),
        # a decode step at up to 128K over the 8-bit pool, batch 4, lengths of their own
        dict(name="attend_step_128k_q8", op="attend", B=4, n=1, len=131072, ragged=11, Hq=64, Hkv=8, d=128, dtype="bf16",
             block=16, bits=8, window=0),
        # a chunk of a 128K prompt
        dict(name="attend_chunk_128k", op="attend", B=1, n=2048, len=131072, ragged=0, Hq=32, Hkv=8, d=128,
             dtype="bf16", block=64, bits=0, window=0),
        # a mixed batch: prompts, short continuations and single tokens over the 8-bit pool, windowed, d = 64
        dict(name="attend_mixed_q8", op="attend", B=9, n=900, len=8192, ragged=5, Hq=24, Hkv=8, d=64, dtype="bf16",
             block=32, bits=8, window=1500),
        # an fp32 prompt
        dict(name="attend_prompt_f32", op="attend", B=2, n=500, len=3001, ragged=0, Hq=8, Hkv=2, d=128, dtype="f32",
             block=128, bits=0, window=0),
    ]


def _logint(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    d = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    op = rng.choice(("append", "store", "attend", "attend"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    B = _logint(rng, 1, 12)
    rope = dict(rot=rng.choice((d, d, d // 2, 32, 24)), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7)
    if op == "append":
        n = rng.choice((1, _logint(rng, 1, 16384 // B)))
        length = _logint(rng, n, 16384)
        return dict(op=op, B=B, n=n, len=length, Tmax=-(-length // 256) * 256, Hq=Hkv * rng.choice((1, 2, 4, 8)),
                    Hkv=Hkv, d=d, dtype=dtype, **rope)
    bits = rng.choice((0, 8, 8))
    block = rng.choice((16, 32, 64, 128))
    if op == "store":
        n = rng.choice((1, _logint(rng, 1, 8192)))
        length = _logint(rng, n, 16384)
        return dict(op=op, B=B, n=n, len=length, ragged=rng.randrange(1, 1000), read=rng.choice((256, length, length)),
                    Hq=Hkv * rng.choice((1, 2, 4, 8)), Hkv=Hkv, d=d, dtype=dtype, block=block, bits=bits, **rope)
    G = rng.choice((1, 2, 3, 4, 5, 6, 8, 16))
    n = rng.choice((1, 1, _logint(rng, 1, 1500)))
    length = _logint(rng, n, 65536 if n < 100 else 16384)
    if dtype == "f32" and n > 1:
        length = max(n, min(length, 3000))
        B = min(B, 2)
    return dict(op=op, B=B, n=n, len=length, ragged=rng.randrange(0, 1000), Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype,
                block=block, bits=bits, window=rng.choice((0, 0, _logint(rng, 1, 4096))))


def _lengths(case):
    """Per sequence: new tokens and length after them.  The first sequence has the case's own n and len, the
    others of a ragged case less."""
    B, n, length, seed = case["B"], case["n"], case["len"], case["ragged"]
    if not seed:
        return [n] * B, [length] * B
    r = random.Random(seed)
    new, lens = [n], [length]
    for _ in range(B - 1):
        m = 1 if r.random() < 0.3 else _logint(r, 1, n)
        new.append(m)
        lens.append(_logint(r, m, length))
    return new, lens


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _norm_weight(g, d, dtype):
    return (1 + 0.2 * _randn(g, d)).to(dtype)


def _rope_inputs(case, g, s):
    d, dtype = case["d"], _DT[case["dtype"]]
    s["wq"] = _norm_weight(g, d, dtype) if case["norm"] else None
    s["wk"] = _norm_weight(g, d, dtype) if case["norm"] else None
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    s["freq"] = (_THETA ** (-2.0 * i / case["rot"])).float()


def _projection(case, g, tokens):
    """q, k and v of `tokens` new tokens as one fused projection writes them: [tokens][Hq + 2 Hkv][d], with a few
    large key channels."""
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    x = _randn(g, tokens, Hq + 2 * Hkv, d)
    x[:, Hq:Hq + Hkv, :: d // 4] *= 8.0
    x = x.to(_DT[case["dtype"]])
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _codes(x):
    """Rows of x (last dimension) as e4m3 codes and exponent bytes."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875)).clamp(-120, 119)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, e):
    return torch.ldexp(codes.float(), (e.to(torch.int32) - 127)[..., None])


def _pool_inputs(case, g, s, lens, cap):
    """A block pool that holds `lens` tokens a sequence in blocks dealt out at random; `cap`: tokens a sequence may grow to."""
    Hkv, d, block, bits, dtype = case["Hkv"], case["d"], case["block"], case["bits"], _DT[case["dtype"]]
    need = [-(-n // block) for n in lens]
    width = -(-cap // block)
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    order = order.cpu()
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    s["table"] = table.cuda()
    shape = (blocks, Hkv, block, d)
    s["K"] = torch.empty(shape, dtype=torch.float8_e4m3fn if bits else dtype, device="cuda")
    s["V"] = torch.empty_like(s["K"])
    s["Ke"] = torch.empty(shape[:3], dtype=torch.uint8, device="cuda") if bits else None
    s["Ve"] = torch.empty_like(s["Ke"]) if bits else None
    for lo in range(0, blocks, 4096):
        hi = min(blocks, lo + 4096)
        for X, E, big in (("K", "Ke", 4.0), ("V", "Ve", 1.0)):
            x = _randn(g, hi - lo, *shape[1:])
            x[..., :: d // 4] *= big
            x = x.to(dtype).float()
            if bits:
                s[X][lo:hi], s[E][lo:hi] = _codes(x)
            else:
                s[X][lo:hi] = x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    s = dict(case=case)
    Hq, Hkv, d, B, dtype = case["Hq"], case["Hkv"], case["d"], case["B"], _DT[case["dtype"]]
    if case["op"] == "append":
        n, Tmax = case["n"], case["Tmax"]
        _rope_inputs(case, g, s)
        q, k, v = _projection(case, g, B * n)
        s["q"], s["k"], s["v"] = (x.unflatten(0, (B, n)).transpose(1, 2) for x in (q, k, v))  # [B][H][n][d] views
        s["lens"] = torch.full((B,), case["len"], dtype=torch.int64, device="cuda")
        s["K"] = torch.zeros(B, Hkv, Tmax, d, dtype=dtype, device="cuda")
        s["V"] = torch.zeros_like(s["K"])
        s["q_out"] = torch.zeros(B, Hq, n, d, dtype=dtype, device="cuda")
        if own:
            from hierarchical_long_context_b200 import api
            s["params"] = api.Params(B=B, Hq=Hq, Hkv=Hkv, d=d, Tmax=Tmax, dtype=dtype)
            s["rope"] = api.Rope(s["freq"], q_norm=s["wq"], k_norm=s["wk"], interleaved=case["interleaved"], eps=_EPS)
        return s
    new, lens = _lengths(case)
    N = sum(new)
    begin = [sum(new[:b]) for b in range(B + 1)]
    s["new"], s["lengths"], s["begin_at"] = new, lens, begin
    s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
    s["begin"] = torch.tensor(begin, dtype=torch.int64, device="cuda")
    _pool_inputs(case, g, s, lens, max(lens))
    if case["op"] == "store":
        _rope_inputs(case, g, s)
        s["q"], s["k"], s["v"] = _projection(case, g, N)
        s["q_out"] = torch.zeros(N, Hq, d, dtype=dtype, device="cuda")
        T = -(-max(lens) // 256) * 256
        s["dense_K"] = torch.zeros(B, Hkv, T, d, dtype=dtype, device="cuda")
        s["dense_V"] = torch.zeros_like(s["dense_K"])
    else:
        s["q"] = (1.5 * _randn(g, N, Hq, d)).to(dtype)
        s["out"] = torch.zeros(N, Hq, d, dtype=dtype, device="cuda")
        s["lse"] = torch.zeros(N, Hq, dtype=torch.float32, device="cuda")
    if own:
        from hierarchical_long_context_b200 import api
        s["pool"] = api.Pool(s["K"], s["V"], s["Ke"], s["Ve"], Hq=Hq, dtype=dtype)
        s["batch"] = api.PoolBatch(s["table"], s["lens"], s["begin"], tokens=N, max_new=max(new))
        if case["op"] == "store":
            s["rope"] = api.Rope(s["freq"], q_norm=s["wq"], k_norm=s["wk"], interleaved=case["interleaved"], eps=_EPS)
        else:
            s["ws"] = api.pool_workspace(s["pool"], s["batch"])
    return s


# ---------------------------------------------------------------- plain forms

def _norm_rotate(case, x, w, pos, freq):
    """fp32: x [..., tokens, d] (tokens' positions `pos`), normed per row and rotated."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()
    rot = case["rot"]
    angle = pos.double()[..., None] * freq.double()
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    y, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((y, rest), -1)


def _plain_append(s):
    case = s["case"]
    n = case["n"]
    pos = s["lens"][:, None] - n + torch.arange(n, device="cuda")  # [B][n]
    s["q_out"].copy_(_norm_rotate(case, s["q"], s["wq"], pos[:, None], s["freq"]))
    k = _norm_rotate(case, s["k"], s["wk"], pos[:, None], s["freq"])
    b = torch.arange(case["B"], device="cuda")[:, None]
    s["K"].transpose(1, 2)[b, pos] = k.transpose(1, 2).to(s["K"].dtype)
    s["V"].transpose(1, 2)[b, pos] = s["v"].transpose(1, 2)
    return {"q": s["q_out"], "K": s["K"], "V": s["V"]}


def _plain_store(s):
    case = s["case"]
    bits, block, dtype = case["bits"], case["block"], _DT[case["dtype"]]
    N, B = s["q"].shape[0], case["B"]
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), s["begin"].diff(), output_size=N)
    pos = s["lens"][seq] - s["begin"][seq + 1] + torch.arange(N, device="cuda")
    s["q_out"].copy_(_norm_rotate(case, s["q"], s["wq"], pos[:, None], s["freq"]))
    k = _norm_rotate(case, s["k"], s["wk"], pos[:, None], s["freq"])
    v = s["v"].float()
    blk, off = s["table"][seq, pos // block].long(), pos % block
    for X, E, x in (("K", "Ke", k), ("V", "Ve", v)):
        if bits:
            code, e = _codes(x)
            s[X].view(torch.uint8).transpose(1, 2)[blk, off] = code.view(torch.uint8)
            s[E].transpose(1, 2)[blk, off] = e
        else:
            s[X].transpose(1, 2)[blk, off] = x.to(dtype)
    # read back the last `read` tokens of every sequence
    T = s["dense_K"].shape[2]
    lo = max(0, case["len"] - case["read"])
    t = torch.arange(lo, case["len"], device="cuda")
    b, t = torch.nonzero(t[None] < s["lens"][:, None], as_tuple=True)
    t = t + lo
    blk, off = s["table"][b, t // block].long(), t % block
    for X, E, Y in (("K", "Ke", "dense_K"), ("V", "Ve", "dense_V")):
        rows = s[X].view(torch.uint8).transpose(1, 2)[blk, off].view(torch.float8_e4m3fn) if bits else s[X].transpose(1, 2)[blk, off]
        if bits:
            rows = _values(rows, s[E].transpose(1, 2)[blk, off]).to(dtype)
        s[Y].transpose(1, 2)[b, t] = rows
    return {"q": s["q_out"], "K": s["dense_K"], "V": s["dense_V"]}


def _rows_of(s, b, X, E):
    """Sequence b's cache rows as fp32 [Hkv][length][d]."""
    case, L = s["case"], s["lengths"][b]
    blk = s["table"][b, : -(-L // case["block"])].long()
    rows = s[X].view(torch.uint8)[blk].view(s[X].dtype)
    rows = _values(rows, s[E][blk]) if case["bits"] else rows.float()
    return rows.transpose(0, 1).flatten(1, 2)[:, :L]


def _plain_attend(s):
    case = s["case"]
    Hq, Hkv, d, window = case["Hq"], case["Hkv"], case["d"], case["window"]
    G = Hq // Hkv
    for b in range(case["B"]):  # every sequence has a length of its own
        n, L, at = s["new"][b], s["lengths"][b], s["begin_at"][b]
        K, V = _rows_of(s, b, "K", "Ke"), _rows_of(s, b, "V", "Ve")
        q = s["q"][at:at + n].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)  # [Hkv][G][n][d]
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        hidden = (key > pos) | ((key <= pos - window) if window else False)
        step = max(1, (1 << 30) // (G * n * L))  # heads whose scores fit 4 GB
        for h in range(0, Hkv, step):
            kv = slice(h, h + step)
            sc = (q[kv].flatten(1, 2) @ K[kv].transpose(1, 2)).unflatten(1, (G, n)) * (1.0 / math.sqrt(d))
            sc = sc.masked_fill_(hidden, -math.inf)
            m = sc.amax(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            o = (p.flatten(1, 2) @ V[kv]).unflatten(1, (G, n)) / total
            heads = slice(h * G, min(Hkv, h + step) * G)
            s["out"][at:at + n, heads] = o.flatten(0, 1).transpose(0, 1).to(s["out"].dtype)
            s["lse"][at:at + n, heads] = (m + total.log())[..., 0].flatten(0, 1).transpose(0, 1)
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    op = s["case"]["op"]
    if own:
        from hierarchical_long_context_b200 import api
        if op == "append":
            api.lod_append_rope(s["params"], s["rope"], s["q"], s["k"], s["v"], s["K"], s["V"], s["lens"],
                                q_out=s["q_out"])
            return {"q": s["q_out"], "K": s["K"], "V": s["V"]}
        if op == "store":
            api.lod_pool_append(s["pool"], s["batch"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
            api.lod_pool_read(s["pool"], s["batch"], s["dense_K"], s["dense_V"],
                              t_begin=max(0, s["case"]["len"] - s["case"]["read"]), t_end=s["case"]["len"])
            return {"q": s["q_out"], "K": s["dense_K"], "V": s["dense_V"]}
        api.lod_pool_attend(s["pool"], s["batch"], s["q"], out=s["out"], lse=s["lse"], window=s["case"]["window"],
                            ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"append": _plain_append, "store": _plain_store, "attend": _plain_attend}[op](s)


# ---------------------------------------------------------------- exact values

def _rotated64(case, x, w, pos, freq):
    """[tokens][heads][d] in fp64: each pair of channels as a complex number turned by its angle."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w.double()
    half = case["rot"] // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * freq.double())
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _e4m3_nearest(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to the even code, from the format's spacing: 2^-9 below
    2^-6, an eighth of the power of two above."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)  # torch.round: ties to even


def _stored64(x):
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(a / 448.0)).clamp(-120, 119)
    e = torch.where((a > 448.0 * torch.exp2(e)) & (e < 119), e + 1, e)
    e = torch.where((a <= 448.0 * torch.exp2(e - 1)) & (e > -120), e - 1, e)
    return _e4m3_nearest(x * torch.exp2(-e)) * torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    dev = "cuda"
    if case["op"] == "append":
        B, n = case["B"], case["n"]
        K, V = s["K"].double(), s["V"].double()
        q = torch.empty(s["q_out"].shape, dtype=torch.float64, device=dev)
        pos = torch.arange(case["len"] - n, case["len"], device=dev)
        for b in range(B):
            q[b] = _rotated64(case, s["q"][b].transpose(0, 1), s["wq"], pos, s["freq"]).transpose(0, 1)
            K[b, :, pos] = _rotated64(case, s["k"][b].transpose(0, 1), s["wk"], pos, s["freq"]).transpose(0, 1)
            V[b, :, pos] = s["v"][b].double()
        return {"q": q, "K": K, "V": V}
    block, bits = case["block"], case["bits"]

    def cached(b, X, E):  # sequence b's rows [length][Hkv][d] in fp64
        L = s["lengths"][b]
        t = torch.arange(L, device=dev)
        blk, off = s["table"][b].long()[t // block], t % block
        rows = s[X].view(torch.uint8 if bits else s[X].dtype).permute(0, 2, 1, 3)[blk, off]
        if not bits:
            return rows.double()
        rows = rows.view(torch.float8_e4m3fn).double()
        return rows * torch.exp2(s[E].permute(0, 2, 1)[blk, off].double() - 127.0)[..., None]

    if case["op"] == "store":
        K, V = s["dense_K"].double(), s["dense_V"].double()
        q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        for b in range(case["B"]):
            n, L, at = s["new"][b], s["lengths"][b], s["begin_at"][b]
            pos = torch.arange(L - n, L, device=dev)
            q[at:at + n] = _rotated64(case, s["q"][at:at + n], s["wq"], pos, s["freq"])
            k = _rotated64(case, s["k"][at:at + n], s["wk"], pos, s["freq"])
            v = s["v"][at:at + n].double()
            lo = max(0, case["len"] - case["read"])
            for X, E, Y, x in (("K", "Ke", K, k), ("V", "Ve", V, v)):
                rows = cached(b, X, E)
                rows[L - n:] = _stored64(x) if bits else x
                if lo < L:
                    Y[b, :, lo:L] = rows[lo:].transpose(0, 1)
        return {"q": q, "K": K, "V": V}
    if work(case)["flops"] > 5e12:
        return None
    G, window = case["Hq"] // case["Hkv"], case["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=dev)
    for b in range(case["B"]):
        n, L, at = s["new"][b], s["lengths"][b], s["begin_at"][b]
        K, V = cached(b, "K", "Ke"), cached(b, "V", "Ve")
        for i0 in range(0, n, 1024):  # query tokens at a time
            i1 = min(n, i0 + 1024)
            last = L - n + i1 - 1
            first = max(0, L - n + i0 - window + 1) if window else 0
            pos = torch.arange(L - n + i0, last + 1, device=dev)[:, None]
            key = torch.arange(first, last + 1, device=dev)[None]
            seen = (key <= pos) & ((key > pos - window) if window else True)
            for h in range(case["Hq"]):
                k, v = K[first:last + 1, h // G], V[first:last + 1, h // G]
                x = torch.where(seen, s["q"][at + i0:at + i1, h].double() @ k.t() / math.sqrt(case["d"]), -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at + i0:at + i1, h] = z
                out[at + i0:at + i1, h] = torch.exp(x - z[:, None]) @ v
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- work

def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        N = case["B"] * case["n"]
        return {"bytes": N * (2 * Hq + 4 * Hkv) * d * e, "flops": N * (Hq + Hkv) * d * 10}
    new, lens = _lengths(case)
    N = sum(new)
    row = d + 1 if case["bits"] else d * e  # a stored row
    if case["op"] == "store":
        lo = max(0, case["len"] - case["read"])
        read = sum(max(0, L - lo) for L in lens)
        return {"bytes": N * (2 * Hq + 2 * Hkv) * d * e + 2 * (N + read) * Hkv * row + 2 * read * Hkv * d * e,
                "flops": N * (Hq + 2 * Hkv) * d * 10 + 2 * read * Hkv * d}
    w = case["window"] or 1 << 60
    pairs = keys = 0
    for n, L in zip(new, lens):
        keys += L - max(0, L - n + 1 - w)
        full = min(max(0, L - max(w, L - n + 1) + 1), n) if w <= L else 0  # queries that see exactly w keys
        m = n - full
        pairs += full * w + m * (L - n) + m * (m + 1) // 2 if full else n * (L - n) + n * (n + 1) // 2
    return {"bytes": 2 * N * Hq * d * e + 4 * N * Hq + 2 * keys * Hkv * row, "flops": 4 * d * Hq * pairs}
