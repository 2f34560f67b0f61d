"""Cases of the serving and training operators around attention over a paged cache.

Three operators, each measured through the calls a program makes:

``norm_rope``  RMS norm of every query and key head with the rotary position embedding, forward
               and backward (``jfa_norm_rope_fwd`` / ``jfa_norm_rope_bwd``).
``cache``      new keys and values written into a paged cache in MXFP8, and read back
               (``jfa_cache_write`` / ``jfa_cache_read``).
``paged``      softmax attention of a chunk of new tokens over the paged cache, with grouped heads
               (``jfa_paged_fwd``); it builds its own work lists in every pass.

With ``own`` false, ``run`` computes the same in elementary torch operations.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 32  # columns that share one scale in the MXFP8 cache


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of each of 256 users in a serving step: latency
        dict(name="norm_rope step", op="norm_rope", dir="fwd", tokens=256, hq=32, hk=8, dim=128,
             rot=128, layout="halves", dtype="bf16", scaling="none", factor=1.0, far=4096),
        # the packed histories of a training batch
        dict(name="norm_rope histories", op="norm_rope", dir="fwd", tokens=131077, hq=32, hk=8, dim=128,
             rot=128, layout="halves", dtype="bf16", scaling="none", factor=1.0, far=4096),
        # fp32 model, part of an odd-sized head rotated, interleaved, stretched to long contexts
        dict(name="norm_rope long f32", op="norm_rope", dir="fwd", tokens=20011, hq=8, hk=8, dim=80,
             rot=48, layout="pairs", dtype="f32", scaling="yarn", factor=16.0, far=1000000),
        # the backward pass of the training batch, with the norms' weight gradients
        dict(name="norm_rope train", op="norm_rope", dir="bwd", tokens=65539, hq=32, hk=8, dim=128,
             rot=64, layout="halves", dtype="bf16", scaling="none", factor=1.0, far=4096),
        # one new token a user written into the cache: latency
        dict(name="cache write step", op="cache", dir="write", batch=256, new_lo=1, new_hi=1, past=4096,
             hk=8, dim=128, dim_v=128, page=64, dtype="bf16"),
        # whole prompts written into the cache
        dict(name="cache write prompts", op="cache", dir="write", batch=64, new_lo=1, new_hi=4096, past=0,
             hk=8, dim=128, dim_v=128, page=64, dtype="bf16"),
        # the cached history read back, to be attended densely or moved elsewhere
        dict(name="cache read", op="cache", dir="read", batch=61, new_lo=1, new_hi=2048, past=1000,
             hk=8, dim=128, dim_v=64, page=16, dtype="bf16"),
        # a few users with short histories, one token each: latency
        dict(name="paged few", op="paged", batch=4, new_lo=1, new_hi=1, len_lo=1, len_hi=700, hq=8, hk=8,
             dim=64, dim_v=64, page=16, cache="bf16", dtype="bf16"),
        # a serving step: one token for each of 256 users over their bf16 caches
        dict(name="paged step", op="paged", batch=256, new_lo=1, new_hi=1, len_lo=1, len_hi=4096, hq=32, hk=8,
             dim=128, dim_v=128, page=64, cache="bf16", dtype="bf16"),
        # a serving step over an MXFP8 cache, longer histories
        dict(name="paged step mxfp8", op="paged", batch=96, new_lo=1, new_hi=2, len_lo=512, len_hi=16384, hq=32,
             hk=4, dim=128, dim_v=128, page=64, cache="mxfp8", dtype="bf16"),
        # chunks of prompts over what is cached of them already
        dict(name="paged chunk mxfp8", op="paged", batch=13, new_lo=1, new_hi=512, len_lo=512, len_hi=16384, hq=32,
             hk=4, dim=128, dim_v=128, page=32, cache="mxfp8", dtype="bf16"),
        # whole prompts of different lengths, causal
        dict(name="paged prompts", op="paged", batch=8, new_lo=1024, new_hi=4096, len_lo=0, len_hi=0, hq=32,
             hk=8, dim=128, dim_v=128, page=128, cache="bf16", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "paged", "paged"])
    if op == "norm_rope":
        dim = rng.choice([32, 48, 64, 80, 96, 128])
        hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), tokens=_log(rng, 100, 60000), hq=hk * rng.choice([1, 2, 3, 4]),
                    hk=hk, dim=dim, rot=16 * rng.randint(1, dim // 16), layout=rng.choice(["halves", "pairs"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 16.0]), far=_log(rng, 1000, 1000000))
    dim, dim_v = rng.choice([(64, 64), (128, 128), (128, 64)])
    page = rng.choice([16, 32, 64, 128])
    if op == "cache":
        return dict(op=op, dir=rng.choice(["write", "read"]), batch=_log(rng, 1, 60), new_lo=1, new_hi=_log(rng, 1, 2000),
                    past=_log(rng, 1, 4000), hk=rng.choice([1, 2, 4, 8]), dim=dim, dim_v=dim_v, page=page,
                    dtype=rng.choice(["bf16", "f32"]))
    hk = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * hk <= 32])
    new_hi = rng.choice([1, 1, 4, _log(rng, 8, 512)])
    batch = _log(rng, 1, 64) if new_hi <= 4 else _log(rng, 1, 8)
    return dict(op=op, batch=batch, new_lo=1, new_hi=new_hi, len_lo=1,
                len_hi=_log(rng, 100, 40000 if new_hi <= 4 else 8000), hq=hk * group,
                hk=hk, dim=dim, dim_v=dim_v, page=page, cache=rng.choice(["bf16", "mxfp8"]), dtype="bf16")


# ------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """New tokens and cached length (the new tokens among it) of every sequence: a fixed ragged
    draw that depends on the case alone."""
    r = random.Random("%(batch)d %(new_lo)d %(new_hi)d %(page)d" % case)
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    if case["op"] == "cache":
        return new, [n + r.randint(0, case["past"]) for n in new]
    return new, [n + r.randint(case["len_lo"], case["len_hi"]) for n in new]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32, device="cuda")


def _quantize(x):
    """MXFP8 codes and biased scale exponents of fp32 rows (last axis in blocks of 32)."""
    b = x.unflatten(-1, (-1, BLOCK))
    f, k = torch.frexp(b.abs().amax(-1))
    e = torch.where(f <= 0.875, k - 9, k - 8).clamp(-100, 119)  # smallest e with amax <= 448 * 2^e
    e = torch.where(f == 0, torch.full_like(e, -100), e)
    y = torch.ldexp(b, -e.unsqueeze(-1))
    return y.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _dequantize(codes, scales):
    y = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK))
    return torch.ldexp(y, scales.int().unsqueeze(-1) - 127).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)
    s = dict(case=case)
    if case["op"] == "norm_rope":
        T, D, n = case["tokens"], case["dim"], case["hq"] + case["hk"]
        # queries and keys are slices of one projection's output; rows of different size
        x = _randn(g, T, n, D).mul_(torch.exp(0.5 * _randn(g, T, 1, 1))).to(dt)
        s.update(q=x[:, :case["hq"]], k=x[:, case["hq"]:], pos=torch.randint(0, case["far"], (T,), generator=g, device="cuda"),
                 wq=1.0 + 0.1 * _randn(g, D), wk=1.0 + 0.1 * _randn(g, D))
        if case["dir"] == "bwd":
            s.update(dyq=_randn(g, T, case["hq"], D).to(dt), dyk=_randn(g, T, case["hk"], D).to(dt))
        return s
    new, lens = _lengths(case)
    B, T, ps, hk = case["batch"], sum(new), case["page"], case["hk"]
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    used = [-(-n // ps) for n in lens]
    width, pages = max(used), sum(used)
    # every sequence's pages lie anywhere in the cache
    order = torch.randperm(pages, generator=g, device="cuda").int()
    n_used = torch.tensor(used, device="cuda")
    first = torch.cumsum(n_used, 0) - n_used
    j = torch.arange(width, device="cuda")
    table = torch.where(j < n_used[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], 0).int().contiguous()
    s.update(offs=torch.tensor(offs, device="cuda"), lens=torch.tensor(lens, device="cuda"), table=table,
             ws=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    kshape, vshape = (pages, hk, ps, case["dim"]), (pages, hk, ps, case["dim_v"])
    if case["op"] == "cache" and case["dir"] == "write":
        s.update(k=_randn(g, T, hk, case["dim"]).to(dt), v=_randn(g, T, hk, case["dim_v"]).to(dt))
        zeros = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        s.update(kc=zeros(*kshape), vc=zeros(*vshape), ks=zeros(*kshape[:3], kshape[3] // BLOCK),
                 vs=zeros(*vshape[:3], vshape[3] // BLOCK))
        return s
    k, v = _randn(g, *kshape), _randn(g, *vshape)
    if case["op"] == "cache" or case["cache"] == "mxfp8":
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _quantize(k), _quantize(v)
    else:
        s.update(kc=k.to(dt), vc=v.to(dt), ks=None, vs=None)
    if case["op"] == "paged":
        s["q"] = _randn(g, T, case["hq"], case["dim"]).to(dt)
    return s


# ------------------------------------------------------------------------------ plain forms
def _theta(case):
    """Rotation frequencies of the pairs, in 64 bits."""
    rot, base, f = case["rot"], 10000.0, case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2))
    theta = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        theta = theta / f
    if case["scaling"] == "yarn":  # a context of 4096 stretched by f, turns between 1 and 32 blended
        keep = ((4096 * theta / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / f)
    return theta


def _amp(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _cos_sin(case, pos):
    a = pos.double()[:, None] * _theta(case)
    return (_amp(case) * torch.cos(a)).float()[:, None], (_amp(case) * torch.sin(a)).float()[:, None]


def _turn(case, x, c, s):
    """The pairs of the first `rot` columns turned by (c, s); the other columns as they are."""
    rot = case["rot"]
    if case["layout"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_norm_rope(case, x, w, c, s):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return _turn(case, x * r * w, c, s).to(_dtype(case))


def _plain_norm_rope_bwd(case, x, w, c, s, dy):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    g = _turn(case, dy.float(), c, -s)
    dw = (g * xh).sum((0, 1), dtype=torch.float64).float()
    g = g * w
    return (r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(_dtype(case)), dw


def _places(s):
    """Of every new token: its row in the cache seen as [pages * page, ...] per head."""
    offs, lens, ps = s["offs"], s["lens"], s["case"]["page"]
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(offs, t, right=True) - 1
    p = lens[b] - (offs[b + 1] - t)
    return s["table"][b, p // ps].long(), p % ps


def _plain_paged(s):
    case, offs, lens = s["case"], s["offs"], s["lens"]
    hq, hk, ps = case["hq"], case["hk"], case["page"]
    new = offs[1:] - offs[:-1]
    n = max(_lengths(case)[0])
    i = torch.arange(n, device="cuda")
    at = (offs[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [B, n] token of every padded row
    q = s["q"][at].float().unflatten(2, (hk, hq // hk))         # [B, n, hk, g, d]
    table = s["table"].long()

    def dense(codes, scales):  # [B, hk, keys, d] in 32 bits
        x = codes[table].float() if scales is None else _dequantize(codes[table], scales[table])
        return x.transpose(1, 2).flatten(2, 3)

    k, v = dense(s["kc"], s["ks"]), dense(s["vc"], s["vs"])
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                  # [B, hk, g n, d]
    x = torch.matmul(q * case["dim"] ** -0.5, k.transpose(2, 3))
    j = torch.arange(k.shape[2], device="cuda")
    seen = j < torch.minimum(lens[:, None], (lens - new)[:, None] + i + 1)[..., None]  # [B, n, keys]
    seen = seen[:, None, None].expand(-1, 1, hq // hk, -1, -1).flatten(2, 3)
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / l
    lse = (m + torch.log(l))[..., 0]
    o = o.unflatten(2, (hq // hk, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, n, hq, dv]
    lse = lse.unflatten(2, (hq // hk, n)).permute(0, 3, 1, 2).flatten(2, 3)
    rows = i < new[:, None]
    return o[rows].to(_dtype(case)), lse[rows]


def _plain(s):
    case = s["case"]
    if case["op"] == "norm_rope":
        c, sn = _cos_sin(case, s["pos"])
        if case["dir"] == "fwd":
            return [_plain_norm_rope(case, s["q"], s["wq"], c, sn), _plain_norm_rope(case, s["k"], s["wk"], c, sn)]
        dq, dwq = _plain_norm_rope_bwd(case, s["q"], s["wq"], c, sn, s["dyq"])
        dk, dwk = _plain_norm_rope_bwd(case, s["k"], s["wk"], c, sn, s["dyk"])
        return [dq, dk, dwq, dwk]
    if case["op"] == "paged":
        return list(_plain_paged(s))
    s["total"] = sum(_lengths(case)[0])
    page, row = _places(s)
    if case["dir"] == "read":
        return [_dequantize(s["kc"][page, :, row], s["ks"][page, :, row]).to(_dtype(case)),
                _dequantize(s["vc"][page, :, row], s["vs"][page, :, row]).to(_dtype(case))]
    s["kc"][page, :, row], s["ks"][page, :, row] = _quantize(s["k"].float())
    s["vc"][page, :, row], s["vs"][page, :, row] = _quantize(s["v"].float())
    return _written(s)


def _written(s):
    return [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn), s["ks"], s["vs"]]


# ------------------------------------------------------------------------------ the framework's calls
def _own(s):
    import jagged_attention_recsys_gb300 as jfa

    case = s["case"]
    if case["op"] == "norm_rope":
        rope = jfa.jfa_rope(case["rot"], layout=case["layout"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                            orig_len=4096, turns_fast=32.0, turns_slow=1.0, amp=_amp(case))
        if case["dir"] == "fwd":
            return list(jfa.jfa_norm_rope_fwd(s["q"], s["k"], s["pos"], s["wq"], s["wk"], rope=rope, eps=EPS))
        return list(jfa.jfa_norm_rope_bwd(s["q"], s["k"], s["pos"], s["dyq"], s["dyk"], s["wq"], s["wk"], rope=rope, eps=EPS))
    cache = jfa.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"])
    if case["op"] == "paged":
        return list(jfa.jfa_paged_fwd(s["q"], cache, s["table"], s["offs"], s["lens"], ws=s["ws"]))
    if case["dir"] == "read":
        if "total" not in s:  # the program knows how many rows it asks for
            s["total"] = sum(_lengths(case)[0])
        return list(jfa.jfa_cache_read(cache, s["table"], s["offs"], s["lens"], s["total"], dtype=_dtype(case), ws=s["ws"]))
    jfa.jfa_cache_write(s["k"], s["v"], cache, s["table"], s["offs"], s["lens"], ws=s["ws"])
    return _written(s)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_rope":
        values = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        fwd = case["dir"] == "fwd"
        return {"bytes": (2 if fwd else 3) * e * values + 8 * case["tokens"] + (8 if fwd else 16) * case["dim"],
                "flops": (8 if fwd else 16) * values}
    new, lens = _lengths(case)
    T, B, d = sum(new), case["batch"], case["dim"] + case["dim_v"]
    index = 8 * (2 * B + 1)
    if case["op"] == "cache":
        pages = sum(-(-n // case["page"]) for n in new)
        return {"bytes": T * case["hk"] * (d * e + d + d // BLOCK) + index + 4 * pages, "flops": 4 * T * case["hk"] * d}
    row = d * e if case["cache"] == "bf16" else d + d // BLOCK
    pages = sum(-(-n // case["page"]) for n in lens)
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, lens))
    return {"bytes": sum(lens) * case["hk"] * row + T * case["hq"] * (d * e + 4) + index + 4 * pages,
            "flops": 2 * pairs * case["hq"] * d}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_norm_rope(case, x, w, pos):
    """One tensor's rows, with complex multiplication for the rotation."""
    rot, f, base = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "ntk":
        base *= f ** (rot / (rot - 2))
    freq = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        turns = 4096 * t / (2 * math.pi)
        if case["scaling"] == "linear":
            t /= f
        elif case["scaling"] == "yarn":
            part = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            t = (1 - part) * t / f + part * t
        freq.append(t)
    ang = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(ang, _amp(case)), ang)[:, None]
    n = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
    if case["layout"] == "halves":
        y = torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * z
        y = torch.cat([y.real, y.imag], -1)
    else:
        y = torch.view_as_real(torch.view_as_complex(n[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    return torch.cat([y, n[..., rot:]], -1)


def _e4m3(y):
    """The nearest e4m3 value, ties to even, in 64 bits: a whole number of steps of the binade."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_rows(x):
    """Codes' values of rows in blocks of 32, in 64 bits."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -140))) - 8
    e = torch.where(a > 448 * torch.exp2(e), e + 1, e).clamp(-100, 119)
    return _e4m3(b / torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        w = [s["wq"].double(), s["wk"].double()]
        x = [s["q"].double(), s["k"].double()]
        if case["dir"] == "fwd":
            return [_exact_norm_rope(case, x[n], w[n], s["pos"]) for n in (0, 1)]
        dx, dw = [], []
        for n, dy in enumerate((s["dyq"], s["dyk"])):
            x[n].requires_grad_(), w[n].requires_grad_()
            a, b = torch.autograd.grad(_exact_norm_rope(case, x[n], w[n], s["pos"]), (x[n], w[n]), dy.double())
            dx.append(a), dw.append(b)
        return dx + dw
    new, lens = _lengths(case)
    ps, table, t0 = case["page"], s["table"].cpu(), 0
    if case["op"] == "cache":
        pages, rows = [], []
        for b, (n, m) in enumerate(zip(new, lens)):
            for p in range(m - n, m):
                pages.append(int(table[b, p // ps])), rows.append(p % ps)
        pages, rows = torch.tensor(pages, device="cuda"), torch.tensor(rows, device="cuda")
        if case["dir"] == "write":
            out = []
            for x, c in ((s["k"], s["kc"]), (s["v"], s["vc"])):
                y = torch.zeros(c.shape, dtype=torch.float64, device="cuda")
                y[pages, :, rows] = _exact_rows(x)
                out.append(y)
            return out + [None, None]
        out = []
        for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            y = c[pages, :, rows].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, BLOCK))
            out.append((y * torch.exp2(sc[pages, :, rows].double() - 127)[..., None]).flatten(-2))
        return out
    group, out_o, out_l = case["hq"] // case["hk"], [], []
    for b, (n, m) in enumerate(zip(new, lens)):
        pages = table[b, :-(-m // ps)].long().cuda()
        kv = []
        for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            y = c[pages]
            if sc is None:
                y = y.double()
            else:
                y = y.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, BLOCK))
                y = (y * torch.exp2(sc[pages].double() - 127)[..., None]).flatten(-2)
            kv.append(y.transpose(0, 1).flatten(1, 2)[:, :m])  # [hk, m, d]
        q = s["q"][t0:t0 + n].double().transpose(0, 1)  # [hq, n, d]
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        o, l = [], []
        for h in range(case["hk"]):
            x = q[h * group:(h + 1) * group] @ kv[0][h].T / math.sqrt(case["dim"])
            x = x.masked_fill(hidden, -math.inf)
            l.append(torch.logsumexp(x, -1))
            o.append(torch.exp(x - l[-1][..., None]) @ kv[1][h])
        out_o.append(torch.cat(o).transpose(0, 1)), out_l.append(torch.cat(l).T)
        t0 += n
    return [torch.cat(out_o), torch.cat(out_l)]
