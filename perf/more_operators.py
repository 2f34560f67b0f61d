"""Cases of windowed attention, of attention over a shared prefix, and of appending to a paged cache.

Four operators, each measured through the calls a program makes:

``window``  causal attention over jagged histories in which a row sees the last ``window`` keys and
            the first ``sinks`` of its sequence: the forward pass, or forward and backward on one
            plan (``jfa_window_plan``, ``jfa_window_fwd``, ``jfa_window_bwd``).
``paged``   the same mask over a paged cache, from one new token a user to chunks of prompts
            (``jfa_paged_window_fwd``).
``append``  RMS norm and rotary positions of new queries and keys, with the keys and values written
            into the cache's pages on the way (``jfa_rope_append``).
``shared``  attention of many short sequences that share a long cached prefix, and have cached keys of
            their own behind it (``jfa_shared_fwd``).

With ``own`` false, ``run`` computes the same in elementary torch operations.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 32  # columns that share one scale in an MXFP8 cache


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of short histories of a small fp32 model, forward and backward: latency
        dict(name="window small f32", op="window", dir="train", batch=4, len_lo=1, len_hi=300, heads=2, dim=32,
             dim_v=32, window=33, sinks=2, dtype="f32"),
        # a training batch's long histories, forward alone (evaluation)
        dict(name="window histories", op="window", dir="fwd", batch=96, len_lo=1, len_hi=4096, heads=8, dim=128,
             dim_v=128, window=512, sinks=4, dtype="bf16"),
        # the training step on such a batch
        dict(name="window train", op="window", dir="train", batch=96, len_lo=1, len_hi=4096, heads=8, dim=128,
             dim_v=128, window=512, sinks=4, dtype="bf16"),
        # one new token of a few users: latency
        dict(name="paged few", op="paged", batch=4, new_lo=1, new_hi=1, len_lo=1, len_hi=700, hq=8, hk=8, dim=64,
             dim_v=64, page=16, window=128, sinks=4, cache="bf16", dtype="bf16"),
        # a serving step: one token for each of 256 users, whose histories are far longer than the window
        dict(name="paged step", op="paged", batch=256, new_lo=1, new_hi=1, len_lo=1, len_hi=8192, hq=32, hk=8,
             dim=128, dim_v=128, page=64, window=1024, sinks=4, cache="bf16", dtype="bf16"),
        # chunks of prompts over an MXFP8 cache
        dict(name="paged chunk mxfp8", op="paged", batch=13, new_lo=1, new_hi=1024, len_lo=512, len_hi=16384, hq=32,
             hk=4, dim=128, dim_v=128, page=32, window=2048, sinks=16, cache="mxfp8", dtype="bf16"),
        # one new token of each of 256 users appended: latency
        dict(name="append step", op="append", batch=256, new_lo=1, new_hi=1, past=4096, hq=32, hk=8, dim=128, dim_v=128,
             rot=128, layout="halves", page=64, cache="bf16", dtype="bf16"),
        # whole prompts appended to an MXFP8 cache
        dict(name="append prompts mxfp8", op="append", batch=64, new_lo=1, new_hi=4096, past=0, hq=32, hk=8, dim=128,
             dim_v=128, rot=128, layout="halves", page=64, cache="mxfp8", dtype="bf16"),
        # an fp32 model with odd heads, part of them rotated in pairs
        dict(name="append f32", op="append", batch=61, new_lo=1, new_hi=700, past=1000, hq=8, hk=8, dim=80, dim_v=64,
             rot=48, layout="pairs", page=16, cache="f32", dtype="f32"),
        # one user's history and eight candidates: latency
        dict(name="shared few", op="shared", groups=1, seqs=8, new_lo=1, new_hi=1, own_lo=0, own_hi=0, prefix_lo=700,
             prefix_hi=700, hq=8, hk=8, dim=64, dim_v=64, page=16, cache="bf16", dtype="bf16"),
        # 16 users, 64 candidates of one to four tokens each scored against the user's history
        dict(name="shared candidates", op="shared", groups=16, seqs=64, new_lo=1, new_hi=4, own_lo=0, own_hi=0,
             prefix_lo=512, prefix_hi=8192, hq=32, hk=8, dim=128, dim_v=128, page=64, cache="bf16", dtype="bf16"),
        # 128 continuations of one long MXFP8 prefix, each with up to 1024 cached tokens of its own, one new token each
        dict(name="shared continuations mxfp8", op="shared", groups=1, seqs=128, new_lo=1, new_hi=1, own_lo=0,
             own_hi=1024, prefix_lo=6011, prefix_hi=6011, hq=32, hk=4, dim=128, dim_v=128, page=64, cache="mxfp8",
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "paged", "append", "shared"])
    dim, dim_v = rng.choice([(64, 64), (128, 128), (128, 64), (64, 128)])
    page = rng.choice([16, 32, 64, 128])
    if op == "window":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            dim, dim_v = rng.choice([8, 32, 40, 64, 100]), rng.choice([8, 32, 40, 64, 100])
        batch, len_hi = _log(rng, 1, 80 if dtype == "bf16" else 12), _log(rng, 4, 4000 if dtype == "bf16" else 600)
        return dict(op=op, dir=rng.choice(["fwd", "train"]), batch=batch, len_lo=0 if batch > 7 else 1, len_hi=len_hi, heads=rng.choice([1, 2, 3, 4, 8]), dim=dim, dim_v=dim_v, window=_log(rng, 1, 5000),
                    sinks=rng.choice([0, 1, 4, 130]), dtype=dtype)
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cache = rng.choice([dtype, "mxfp8"])
        dim = rng.choice([32, 64, 96, 128] if cache == "mxfp8" else [24, 32, 48, 64, 80, 96, 128])
        hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, batch=_log(rng, 1, 60), new_lo=1, new_hi=_log(rng, 1, 2000), past=_log(rng, 1, 4000),
                    hq=hk * rng.choice([1, 2, 3, 4]), hk=hk, dim=dim, dim_v=rng.choice([32, 64, 128]),
                    rot=2 * rng.randint(1, dim // 2), layout=rng.choice(["halves", "pairs"]), page=page, cache=cache,
                    dtype=dtype)
    hk = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * hk <= 32])
    cache = rng.choice(["bf16", "mxfp8"])
    if op == "paged":
        new_hi = rng.choice([1, 1, 4, _log(rng, 8, 900)])
        few = new_hi <= 4
        return dict(op=op, batch=_log(rng, 1, 64) if few else _log(rng, 1, 10), new_lo=1, new_hi=new_hi, len_lo=1,
                    len_hi=_log(rng, 50, 20000 if few else 8000), hq=hk * group, hk=hk, dim=dim, dim_v=dim_v, page=page,
                    window=_log(rng, 1, 4000), sinks=rng.choice([0, 1, 4, 16, 150]), cache=cache, dtype="bf16")
    prefix = _log(rng, 20, 8000)
    return dict(op=op, groups=_log(rng, 1, 12), seqs=_log(rng, 1, 60), new_lo=1, new_hi=rng.choice([1, 1, 3, 20]), own_lo=0,
                own_hi=rng.choice([0, 0, _log(rng, 1, 500)]), prefix_lo=prefix // 2, prefix_hi=prefix, hq=hk * group, hk=hk,
                dim=dim, dim_v=dim_v, page=page, cache=cache, dtype="bf16")


# ------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _shape(case):
    """The batch's lengths: a fixed ragged draw that depends on the case alone.  (new tokens, cached
    lengths with the new tokens among them, prefix lengths, sequences of every group)"""
    r = random.Random("%s %s" % (case["op"], sorted((k, v) for k, v in case.items() if k.endswith(("_lo", "_hi", "seqs")))))
    if case["op"] == "window":
        return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])], None, None, None
    if case["op"] == "shared":
        groups = [case["seqs"]] * case["groups"]
        prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in groups]
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(sum(groups))]
        return new, [n + r.randint(case["own_lo"], case["own_hi"]) for n in new], prefix, groups
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    lo, hi = (case["len_lo"], case["len_hi"]) if case["op"] == "paged" else (0, case["past"])
    return new, [n + r.randint(lo, hi) for n in new], None, None


def _sums(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


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


def _tables(g, lens, page, taken=0):
    """Page table of sequences whose pages lie anywhere in the cache."""
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used), generator=g, device="cuda") + taken
    width = max(max(used), 1)
    n_used = torch.tensor(used, device="cuda")
    first = torch.cumsum(n_used, 0) - n_used
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp(max=max(sum(used) - 1, 0))
    rows = order[at] if sum(used) else torch.zeros_like(at)
    return torch.where(j < n_used[:, None], rows, 0).int().contiguous(), sum(used)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, dv = _dtype(case), case["dim"], case["dim_v"]
    new, lens, prefix, groups = _shape(case)
    T = sum(new)
    s = dict(case=case, total=T, offs=torch.tensor(_sums(new), device="cuda"))
    if case["op"] == "window":
        H = case["heads"]
        s.update(q=_randn(g, T, H, d).to(dt), k=_randn(g, T, H, d).to(dt), v=_randn(g, T, H, dv).to(dt),
                 do=_randn(g, T, H, dv).to(dt))
        return s
    hq, hk, ps = case["hq"], case["hk"], case["page"]
    s["lens"] = torch.tensor(lens, device="cuda")
    s["table"], pages = _tables(g, lens, ps)
    if case["op"] == "append":
        # queries, keys and values are slices of one projection's output; tokens of different size
        x = _randn(g, T, (hq + hk) * d + hk * dv).mul_(torch.exp(0.5 * _randn(g, T, 1))).to(dt)
        a, b = hq * d, (hq + hk) * d
        s.update(q=x[:, :a].unflatten(1, (hq, d)), k=x[:, a:b].unflatten(1, (hk, d)), v=x[:, b:].unflatten(1, (hk, dv)),
                 wq=1.0 + 0.1 * _randn(g, d), wk=1.0 + 0.1 * _randn(g, d))
        mx = case["cache"] == "mxfp8"
        new_ = lambda n, t: torch.zeros(pages, hk, ps, n, dtype=t, device="cuda")  # noqa: E731
        u = torch.uint8
        s.update(kc=new_(d, u if mx else dt), vc=new_(dv, u if mx else dt), ks=new_(d // BLOCK, u) if mx else None,
                 vs=new_(dv // BLOCK, u) if mx else None)
        return s
    if case["op"] == "shared":
        s["prefix_lens"] = torch.tensor(prefix, device="cuda")
        s["prefix_table"], more = _tables(g, prefix, ps, pages)
        s["groups"] = torch.tensor(_sums(groups), device="cuda")
        pages += more
    s["q"] = _randn(g, T, hq, d).to(dt)
    k, v = _randn(g, pages, hk, ps, d), _randn(g, pages, hk, ps, dv)
    if case["cache"] == "mxfp8":
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _quantize(k), _quantize(v)
    else:
        s.update(kc=k.to(dt), vc=v.to(dt), ks=None, vs=None)
    return s


# ------------------------------------------------------------------------------ plain forms
def _softmax(x):
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    return x.div_(torch.where(l == 0, 1.0, l)), (m + torch.log(l))[..., 0]


def _padded(s):
    """The new tokens' rows, padded to the longest sequence: [B, n] tokens, and which exist."""
    offs = s["offs"]
    n = offs[1:] - offs[:-1]
    i = torch.arange(max(max(_shape(s["case"])[0]), 1), device="cuda")
    return (offs[:-1, None] + i).clamp(max=s["total"] - 1), i < n[:, None]


def _plain_window(s):
    case, dt, train = s["case"], _dtype(s["case"]), s["case"]["dir"] == "train"
    names = ["v", "q", "k", "v"][:4 if train else 1]
    out = [torch.empty_like(s[n], memory_format=torch.contiguous_format) for n in names]
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    if s["total"] == 0:
        return out[:1] + [lse] + out[1:]
    at, there = _padded(s)
    i = torch.arange(at.shape[1], device="cuda")
    gap = i[:, None] - i
    hidden = (gap < 0) | ((gap >= case["window"]) & (i >= case["sinks"]))
    scale = case["dim"] ** -0.5
    for h in range(case["heads"]):  # a head at a time: the scores of all would not fit
        q, k, v, do = (torch.where(there[..., None], s[n][at, h].float(), 0.0) for n in ("q", "k", "v", "do"))
        p, z = _softmax(torch.matmul(q * scale, k.transpose(1, 2)).masked_fill_(hidden, -math.inf))
        o = torch.matmul(p, v)
        got = [o]
        if train:
            ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
            got += [torch.matmul(ds, k) * scale, torch.matmul(ds.transpose(1, 2), q) * scale,
                    torch.matmul(p.transpose(1, 2), do)]
        lse[:, h] = z[there]
        for x, y in zip(out, got):
            x[:, h] = y[there].to(dt)
    return out[:1] + [lse] + out[1:]


def _cached(s, table, pos):
    """Keys and values [B, hk, positions, dim] at positions [B, n] of sequences' tables, in 32 bits."""
    ps = s["case"]["page"]
    page, row = torch.gather(table, 1, (pos // ps).clamp(max=table.shape[1] - 1)).long(), pos % ps
    both = []
    for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = c[page, :, row]
        x = x.float() if sc is None else _dequantize(x, sc[page, :, row])
        both.append(x.transpose(1, 2))
    return both


def _heads(s, x):
    """[B, n, hq, d] rows as [B, hk, group n, d], scaled, in 32 bits."""
    hk, g, d = s["case"]["hk"], s["case"]["hq"] // s["case"]["hk"], s["case"]["dim"]
    return x.float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3) * d ** -0.5


def _tokens(s, x):
    """[B, hk, group n, ...] back to [B, n, hq, ...]."""
    g = s["case"]["hq"] // s["case"]["hk"]
    return x.unflatten(2, (g, -1)).flatten(1, 2).transpose(1, 2)


def _plain_paged(s):
    case, lens = s["case"], s["lens"][:, None]
    new, cached, _, _ = _shape(case)
    at, there = _padded(s)
    i = lens - there.sum(1, keepdim=True) + torch.arange(at.shape[1], device="cuda")  # positions of the rows
    low = (i[:, :1] - case["window"] + 1).clamp(min=0)
    wide = min(max(cached), max(new) + case["window"] - 1)
    front = torch.arange(min(case["sinks"], max(cached)), device="cuda").expand(len(new), -1)
    pos = torch.cat([front, low + torch.arange(wide, device="cuda")], 1)
    is_front = torch.arange(pos.shape[1], device="cuda") < front.shape[1]
    k, v = _cached(s, s["table"], pos)
    gap = i[..., None] - pos[:, None]
    sees = torch.where(is_front, pos[:, None] < low[..., None], (gap < case["window"]) | (pos[:, None] < case["sinks"]))
    hidden = ~(sees & (gap >= 0)).repeat(1, case["hq"] // case["hk"], 1)[:, None]
    p, lse = _softmax(torch.matmul(_heads(s, s["q"][at]), k.transpose(2, 3)).masked_fill_(hidden, -math.inf))
    return [_tokens(s, torch.matmul(p, v))[there].to(_dtype(case)), _tokens(s, lse)[there]]


def _plain_shared(s):
    case, G = s["case"], s["case"]["groups"]
    _, cached, prefix, _ = _shape(case)
    at, there = _padded(s)
    q = _heads(s, s["q"][at])  # [B, hk, rows, d]
    B, hk, rows, d = q.shape
    pos = torch.arange(max(prefix), device="cuda")
    k, v = _cached(s, s["prefix_table"], pos.expand(G, -1))
    qg = q.unflatten(0, (G, -1)).transpose(1, 2).flatten(2, 3)  # [G, hk, seqs rows, d]
    x = torch.matmul(qg, k.transpose(2, 3)).masked_fill_((pos >= s["prefix_lens"][:, None])[:, None, None], -math.inf)
    x = x.unflatten(2, (-1, rows)).transpose(1, 2).flatten(0, 1)  # [B, hk, rows, prefix]
    own = torch.arange(max(cached), device="cuda")
    k1, v1 = _cached(s, s["table"], own.expand(B, -1))
    i = s["lens"][:, None] - there.sum(1, keepdim=True) + torch.arange(at.shape[1], device="cuda")
    hidden = (own > i[..., None]).repeat(1, case["hq"] // case["hk"], 1)[:, None]
    y = torch.matmul(q, k1.transpose(2, 3)).masked_fill_(hidden, -math.inf)
    p, lse = _softmax(torch.cat([x, y], -1))
    pg = p[..., :len(pos)].unflatten(0, (G, -1)).transpose(1, 2).flatten(2, 3)
    o = torch.matmul(pg, v).unflatten(2, (-1, rows)).transpose(1, 2).flatten(0, 1) + torch.matmul(p[..., len(pos):], v1)
    return [_tokens(s, o)[there].to(_dtype(case)), _tokens(s, lse)[there]]


def _places(s):
    """Of every new token: its position, page and row in the cache."""
    offs, lens, ps = s["offs"], s["lens"], s["case"]["page"]
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(offs, t, right=True) - 1
    p = lens[b] - (offs[b + 1] - t)
    return p, s["table"][b, p // ps].long(), p % ps


def _turned(case, x, w, pos):
    """Rows normalised, weighted, and their first `rot` columns turned, in 32 bits."""
    rot = case["rot"]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    ang = (pos.double()[:, None] * 10000.0 ** (-2.0 * i / rot))[:, None]
    c, sn = torch.cos(ang).float(), torch.sin(ang).float()
    if case["layout"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    case = s["case"]
    pos, page, row = _places(s)
    yq = _turned(case, s["q"], s["wq"], pos).to(_dtype(case))
    yk = _turned(case, s["k"], s["wk"], pos)
    if case["cache"] == "mxfp8":
        s["kc"][page, :, row], s["ks"][page, :, row] = _quantize(yk)
        s["vc"][page, :, row], s["vs"][page, :, row] = _quantize(s["v"].float())
    else:
        s["kc"][page, :, row], s["vc"][page, :, row] = yk.to(_dtype(case)), s["v"]
    return [yq] + _written(s)


def _written(s):
    """The cache's contents: values, or codes and scales as the numbers they stand for."""
    if s["ks"] is None:
        return [s["kc"], s["vc"]]
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return [s["kc"].view(e4), s["vc"].view(e4), s["ks"].view(e8), s["vs"].view(e8)]


# ------------------------------------------------------------------------------ the framework's calls
def _own(s):
    import jagged_attention_recsys_gb300 as jfa

    case = s["case"]
    if case["op"] == "window":
        q, k, v, offs, w, n = s["q"], s["k"], s["v"], s["offs"], case["window"], case["sinks"]
        if case["dir"] == "fwd":
            return list(jfa.jfa_window_fwd(q, k, v, offs, w, sinks=n))
        ws = jfa.jfa_window_plan(q, k, v, offs, w, sinks=n)
        o, lse = jfa.jfa_window_fwd(q, k, v, offs, w, sinks=n, ws=ws, planned=True)
        return [o, lse, *jfa.jfa_window_bwd(q, k, v, o, lse, s["do"], offs, w, sinks=n, ws=ws, planned=True)]
    cache = jfa.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"])
    if case["op"] == "paged":
        return list(jfa.jfa_paged_window_fwd(s["q"], cache, s["table"], s["offs"], s["lens"], case["window"],
                                             sinks=case["sinks"]))
    if case["op"] == "shared":
        return list(jfa.jfa_shared_fwd(s["q"], cache, s["table"], s["offs"], s["lens"], s["prefix_table"],
                                       s["prefix_lens"], s["groups"]))
    rope = jfa.jfa_rope(case["rot"], layout=case["layout"])
    yq, _ = jfa.jfa_rope_append(s["q"], s["k"], s["v"], cache, s["table"], s["offs"], s["lens"], s["wq"], s["wk"],
                                rope=rope, eps=EPS)
    return [yq] + _written(s)


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "paged": _plain_paged, "append": _plain_append, "shared": _plain_shared}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------------------ work
def _pairs(n, m, window, sinks):
    """Visible pairs of the last n of m positions: keys of row i are min(i + 1, window) of the window and
    the sinks in front of it."""
    total = 0
    for i in range(m - n, m):
        low = max(0, i + 1 - window)
        total += i + 1 - low + min(low, sinks)
    return total


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    new, lens, prefix, groups = _shape(case)
    T, d, dv = sum(new), case["dim"], case["dim_v"]
    if case["op"] == "window":
        H, pairs = case["heads"], sum(_pairs(n, n, case["window"], case["sinks"]) for n in new)
        train = case["dir"] == "train"
        values = T * H * (3 * (d + dv) + d + dv if train else 2 * (d + dv))
        return {"bytes": values * e + 4 * T * H + 8 * (len(new) + 1),
                "flops": pairs * H * 2 * ((d + dv) + (3 * d + 2 * dv if train else 0))}
    hq, hk, ps = case["hq"], case["hk"], case["page"]
    row = d + dv + (d + dv) // BLOCK if case["cache"] == "mxfp8" else (d + dv) * e
    index = 8 * (2 * len(new) + 1)
    if case["op"] == "append":
        return {"bytes": T * (hq * d * 2 + hk * (d + dv)) * e + T * hk * row + index + 8 * d
                + 4 * sum(-(-n // ps) for n in new), "flops": 8 * T * (hq + hk) * d}
    rows = T * hq * ((d + dv) * e + 4)
    if case["op"] == "paged":
        w, n0 = case["window"], case["sinks"]
        keys = pairs = 0
        for n, m in zip(new, lens):
            low = max(0, m - n + 1 - w)
            keys += m - low + min(low, n0)
            pairs += _pairs(n, m, w, n0)
        return {"bytes": keys * hk * row + rows + index + 4 * (keys // ps + len(new)), "flops": 2 * pairs * hq * (d + dv)}
    keys = sum(prefix) + sum(lens)
    first, pairs = _sums(groups), 0
    for g, p in enumerate(prefix):
        pairs += sum(n * (p + m - n) + n * (n + 1) // 2
                     for n, m in zip(new[first[g]:first[g + 1]], lens[first[g]:first[g + 1]]))
    return {"bytes": keys * hk * row + rows + index + 8 * (2 * len(prefix) + 1) + 4 * (keys // ps + len(new)),
            "flops": 2 * pairs * hq * (d + dv)}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_rows(s, table, m):
    """The first m cached rows of one sequence, [hk, m, dim] in 64 bits, page by page."""
    pages = table[:-(-m // s["case"]["page"])].long()
    both = []
    for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        y = c[pages]
        if sc is None:
            y = y.double()
        else:
            y = y.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, BLOCK))
            y = (y * torch.exp2(sc[pages].double() - 127)[..., None]).flatten(-2)
        both.append(y.transpose(0, 1).flatten(1, 2)[:, :m])
    return both


def _attend(q, k, v, hidden):
    """Of [.., n, d] queries: outputs and the log of the sum."""
    x = (q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])).masked_fill(hidden, -math.inf)
    return torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)


def _exact_attention(s):
    case, o, l = s["case"], [], []
    new, lens, prefix, groups = _shape(case)
    group, t0, b = case["hq"] // case["hk"], 0, 0
    for g in range(len(groups) if groups else 1):
        front = _exact_rows(s, s["prefix_table"][g], prefix[g]) if groups else None
        for _ in range(groups[g] if groups else len(new)):
            n, m = new[b], lens[b]
            k, v = _exact_rows(s, s["table"][b], m)
            i, j = torch.arange(m - n, m, device="cuda")[:, None], torch.arange(m, device="cuda")[None]
            hidden = j > i
            if groups:
                k, v = torch.cat([front[0], k], 1), torch.cat([front[1], v], 1)
                hidden = torch.cat([torch.zeros(n, prefix[g], dtype=torch.bool, device="cuda"), hidden], 1)
            else:
                hidden = hidden | ((j <= i - case["window"]) & (j >= case["sinks"]))
            q = s["q"][t0:t0 + n].double().transpose(0, 1).unflatten(0, (case["hk"], group))
            y, z = _attend(q, k[:, None], v[:, None], hidden)
            o.append(y.flatten(0, 1).transpose(0, 1)), l.append(z.flatten(0, 1).T)
            t0, b = t0 + n, b + 1
    return [torch.cat(o), torch.cat(l)]


def _exact_window(s):
    case, out, t0 = s["case"], [], 0
    for n in _shape(case)[0]:
        x = [s[name][t0:t0 + n].double().transpose(0, 1).requires_grad_() for name in "qkv"]
        i = torch.arange(n, device="cuda")
        gap = i[:, None] - i[None]
        o, lse = _attend(*x, (gap < 0) | ((gap >= case["window"]) & (i[None] >= case["sinks"])))
        one = [o.detach().transpose(0, 1), lse.detach().T]
        if case["dir"] == "train":
            grads = torch.autograd.grad(o, x, s["do"][t0:t0 + n].double().transpose(0, 1)) if n else x
            one += [y.detach().transpose(0, 1) for y in grads]
        out.append(one)
        t0 += n
    return [torch.cat(y) for y in zip(*out)]


def _e4m3(y):
    """The nearest e4m3 value, ties to even, in 64 bits: a whole number of steps of the binade."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _coded(x):
    """Codes' values and scales of rows in blocks of 32, in 64 bits."""
    b = x.unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -140))) - 8
    scale = torch.exp2(torch.where(a > 448 * torch.exp2(e), e + 1, e).clamp(-100, 119))
    return _e4m3(b / scale).flatten(-2), scale[..., 0]


def _exact_append(s):
    case = s["case"]
    new, lens, _, _ = _shape(case)
    table, ps, rot = s["table"].cpu(), case["page"], case["rot"]
    pos, pages = [], []
    for b, (n, m) in enumerate(zip(new, lens)):
        pos += range(m - n, m)
        pages += [int(table[b, p // ps]) for p in range(m - n, m)]
    pos, pages = torch.tensor(pos, device="cuda"), torch.tensor(pages, device="cuda")
    ang = pos.double()[:, None] * torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64,
                                               device="cuda")
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    out = []
    for x, w in ((s["q"].double(), s["wq"].double()), (s["k"].double(), s["wk"].double())):
        n = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
        if case["layout"] == "halves":
            y = torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * z
            y = torch.cat([y.real, y.imag], -1)
        else:
            y = torch.view_as_real(torch.view_as_complex(n[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        out.append(torch.cat([y, n[..., rot:]], -1))
    rows = [out[1], s["v"].double()]
    arrays = [s["kc"], s["vc"]]
    if case["cache"] == "mxfp8":
        rows = [y[n] for n in (0, 1) for y in map(_coded, rows)]
        arrays += [s["ks"], s["vs"]]
    cached = [torch.zeros(c.shape, dtype=torch.float64, device="cuda") for c in arrays]
    for c, y in zip(cached, rows):
        c[pages, :, pos % ps] = y
    return [out[0]] + cached


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(s)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
