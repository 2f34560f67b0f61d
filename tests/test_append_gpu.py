"""Norm, rotation and the write to a paged cache in one pass (jfa_rope_append) against plain 64-bit
implementations, and the runs of it with the attention that reads the cache.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref
import window_ref as wref
from test_norm_rope_gpu import FWD, f64, rope_of

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A cache full of a marker, sequences on random pages, and new tokens as slices of one projection."""

    def __init__(self, new, lens, hq, hk, dqk, dv, page, cache, dtype, seed=0, spread=1.0, pad=0):
        rng = np.random.default_rng(seed)
        self.new, self.lens_h = np.array(new, np.int64), np.array(lens, np.int64)
        self.offs_h = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)
        self.B, self.T, self.page, self.dtype, self.hk = len(new), int(self.offs_h[-1]), page, dtype, hk
        used = [-(-int(n) // page) for n in lens]
        self.pages = sum(used) + 2
        order = rng.permutation(self.pages)
        self.table_h = np.full((self.B, max(used + [1])), -1, np.int64)
        at = 0
        for b, n in enumerate(used):
            self.table_h[b, :n] = order[at:at + n]
            at += n
        dev = lambda a, t: torch.tensor(a, dtype=t, device="cuda")
        self.offs, self.lens, self.table = dev(self.offs_h, torch.int64), dev(self.lens_h, torch.int64), dev(self.table_h, torch.int32)
        self.cache = jfa.paged_cache(self.pages, hk, dqk, dv, page_size=page, dtype=DT[dtype], mxfp8=cache == "mxfp8")
        for x in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if x is not None:
                x.fill_(119)
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *n: torch.randn(n, generator=g, device="cuda")
        x = (r(self.T, (hq + hk) * dqk + hk * dv + pad) * torch.exp(spread * r(self.T, 1))).to(DT[dtype])
        a, b = hq * dqk, (hq + hk) * dqk
        self.x = x
        self.q = x[:, :a].unflatten(1, (hq, dqk)) if hq else None
        self.k, self.v = x[:, a:b].unflatten(1, (hk, dqk)), x[:, b:b + hk * dv].unflatten(1, (hk, dv))
        self.wq, self.wk = 1 + 0.1 * r(dqk), 1 + 0.1 * r(dqk)
        self.at = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)] + [np.zeros(0)]).astype(np.int64)
        self.seq = np.repeat(np.arange(self.B), self.new)

    def args(self):
        return self.q, self.k, self.v, self.cache, self.table, self.offs, self.lens

    def space(self, hq=None):
        return jfa.paged_workspace(jfa.paged_params(self.cache, self.table, self.offs, self.lens, self.T, DT[self.dtype],
                                                    heads_q=hq))


def check(c, rot, layout, kw, norm=True, weights=True, pos=None, eps=1e-5, ws=None, **more):
    rope, freq, amp = rope_of(rot, layout, kw)
    rot = 0 if rope is None else rot
    w = dict(wq=c.wq if c.q is not None else None, wk=c.wk) if norm and weights else {}
    c0 = [None if x is None else x.clone() for x in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)]
    q_before = None if c.q is None else f64(c.q)
    ws = c.space(None if c.q is None else c.q.shape[1]) if ws is None else ws
    yq, _ = jfa.jfa_rope_append(*c.args(), rope=rope, eps=eps, norm=norm, pos=pos, ws=ws, **w, **more)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    at = f64(pos) if pos is not None else c.at
    made = lambda x, wt: ref.norm_rope(x, f64(wt) if w else None, at, freq, rot, layout, amp, eps, norm=norm)
    if c.q is not None:
        want, size = made(q_before, c.wq)
        err = np.abs(f64(yq) - want)
        assert np.all(err <= ref.HALF_STEP[c.dtype] * np.abs(want) * 1.01 + FWD * size + 1e-36)
    else:
        assert yq is None
    # the cache: rows of the new tokens at their places, everything else as it was
    live = c.at >= 0
    page, row = c.table_h[c.seq[live], c.at[live] // c.page], c.at[live] % c.page
    other = np.ones((c.pages, c.page), bool)
    other[page, row] = False
    other = torch.tensor(other, device="cuda")[:, None, :, None].expand(-1, c.hk, -1, -1)
    for x, y in zip((c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale), c0):
        if x is not None:
            m = other.expand(x.shape)
            assert torch.equal(x[m], y[m])
    if not live.any():
        return yq
    for name, arr, sc, want, size in (("k", c.cache.k, c.cache.k_scale, *made(f64(c.k), c.wk)),
                                      ("v", c.cache.v, c.cache.v_scale, f64(c.v), None)):
        want = want[live]
        if not c.cache.mxfp8:
            got = f64(arr)[page, :, row]
            if size is None:
                assert np.array_equal(got, want)
            else:
                assert np.all(np.abs(got - want) <= ref.HALF_STEP[c.dtype] * np.abs(want) * 1.01 + FWD * size[live] + 1e-36)
            continue
        codes, exps = arr.cpu().numpy()[page, :, row], sc.cpu().numpy()[page, :, row].astype(np.int64) - 127
        got = ref.decode(codes, (exps + 127).astype(np.uint8))
        val, _, e = ref.quantize_rows(want)
        if size is None:
            assert np.array_equal(exps, e) and np.array_equal(got, val)
            continue
        # the scale is the smallest for the largest value, which is known to a few fp32 roundings
        top = np.abs(want).reshape(want.shape[:-1] + (-1, 32)).max(-1)
        reach = size[live].reshape(want.shape[:-1] + (-1, 32)).max(-1)
        near = np.abs(top / np.ldexp(448.0, np.where(exps < e, exps, e)) - 1) <= 2 * FWD * reach / np.maximum(top, 1e-300)
        assert np.all((exps == e) | ((np.abs(exps - e) == 1) & near))
        # a code is within half a step of its value over the scale: 2^-4 of it, 2^-10 near zero
        step = np.repeat(np.ldexp(1.0, exps), 32, axis=-1)
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want) * 1.01, 2.0 ** -10 * step) + FWD * size[live])
    return yq


EDGES = [0, 1, 15, 16, 17, 31, 33, 64, 100]
CASES = [
    # hq, hk, dqk, dv, rot, layout, page, cache, dtype, rope's arguments
    (4, 2, 64, 64, 64, "halves", 16, "bf16", "bf16", {}),
    (4, 2, 128, 128, 128, "halves", 64, "bf16", "bf16", {}),
    (8, 2, 128, 64, 64, "pairs", 32, "bf16", "bf16", dict(amp=1.1)),
    (32, 4, 128, 128, 128, "halves", 64, "mxfp8", "bf16", {}),
    (3, 1, 64, 128, 32, "halves", 16, "mxfp8", "bf16", {}),
    (2, 2, 96, 32, 48, "halves", 16, "mxfp8", "bf16", {}),
    (2, 2, 96, 96, 80, "halves", 128, "mxfp8", "bf16", {}),
    (6, 3, 96, 64, 96, "pairs", 32, "mxfp8", "bf16", {}),
    (2, 1, 256, 256, 256, "halves", 16, "mxfp8", "bf16", {}),
    (8, 8, 80, 64, 48, "pairs", 16, "f32", "f32", dict(scaling="yarn", factor=16.0, orig_len=4096)),
    (2, 2, 256, 128, 128, "halves", 16, "f32", "f32", {}),
    (4, 1, 64, 64, 64, "halves", 256, "mxfp8", "f32", dict(scaling="ntk", factor=4.0)),
    (3, 3, 32, 32, 16, "pairs", 16, "mxfp8", "f32", {}),
    (2, 2, 40, 24, 40, "halves", 16, "bf16", "bf16", {}),
    (2, 1, 24, 8, 6, "pairs", 16, "f32", "f32", {}),
    (2, 2, 64, 96, 34, "halves", 32, "mxfp8", "bf16", {}),
    (5, 1, 64, 64, 2, "pairs", 32, "mxfp8", "f32", {}),
    (2, 2, 64, 64, 64, "halves", 16, "bf16", "bf16", None),
    (0, 2, 128, 128, 128, "halves", 16, "mxfp8", "bf16", {}),
    (0, 2, 72, 8, 72, "pairs", 16, "bf16", "bf16", {}),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("kind", ["step", "chunk", "prompts"])
@pytest.mark.parametrize("case", CASES, ids=["%d-%d-D%d-%d-r%d-%s-p%d-%s-%s" % c[:9] for c in CASES])
def test_append(case, kind, norm):
    hq, hk, dqk, dv, rot, layout, page, cache, dtype, kw = case
    if kind == "step":
        new, lens = [1] * 9, [n + 1 for n in EDGES]
    elif kind == "chunk":  # some before the cache's start
        new, lens = EDGES, [max(0, n + d) for n, d in zip(EDGES, [0, 70, -3, 5, 0, 300, -33, 1, 40])]
    else:
        new, lens = [700, 0, 301], [700, 0, 301]
    c = Case(new, lens, hq, hk, dqk, dv, page, cache, dtype)
    check(c, rot, layout, kw, norm=norm)


def test_many_tokens_and_sequences():
    rng = np.random.default_rng(1)
    new = rng.integers(0, 60, 900)
    c = Case(new, new + rng.integers(0, 50, 900), 4, 2, 64, 64, 16, "mxfp8", "bf16")
    check(c, 64, "halves", {})
    c = Case([1] * 1500, rng.integers(1, 90, 1500), 8, 1, 128, 128, 16, "bf16", "bf16")
    check(c, 128, "halves", {})


def test_positions_that_are_not_the_caches():
    c = Case([5, 30], [60, 30], 2, 2, 64, 64, 16, "mxfp8", "bf16")
    pos = torch.randint(-1000, 10 ** 6, (c.T,), device="cuda")
    check(c, 64, "pairs", {}, pos=pos)


def test_sizes_at_the_ends_of_the_scales():
    """Keys and values whose blocks meet the smallest and the largest scale, zeros among them."""
    for dtype in ("bf16", "f32"):
        c = Case([40, 7], [40, 20], 2, 2, 64, 64, 16, "mxfp8", dtype)
        k, v = torch.zeros_like(c.k), torch.zeros_like(c.v)
        s = torch.ldexp(torch.ones(c.T, device="cuda"), torch.linspace(-120, 118, c.T, device="cuda").int())
        k[:, 0], v[:, 1] = (c.k[:, 0].float().sign() * s[:, None]).to(k.dtype), (c.v[:, 1].float().sign() * s[:, None]).to(v.dtype)
        c.k, c.v = k, v
        check(c, 64, "halves", {}, norm=False)


def test_in_place_strides_plans_and_given_outputs():
    for cache, dtype, pad in (("bf16", "bf16", 8), ("mxfp8", "bf16", 24), ("f32", "f32", 4)):
        c = Case([3, 50], [9, 50], 4, 2, 64, 64, 16, cache, dtype, pad=pad)
        ws = c.space(4)
        kept = c.x.clone()
        jfa.jfa_paged_plan(c.q, c.cache, c.table, c.offs, c.lens, ws=ws)
        y = check(c, 64, "halves", {}, ws=ws, planned=True, yq=c.q)
        assert y is c.q
        a = 4 * 64
        assert torch.equal(kept[:, a:], c.x[:, a:])  # keys, values and what lies behind them


def test_captured_and_replayed_on_a_stream_of_its_own():
    c = Case([1] * 5, [3, 70, 16, 17, 200], 4, 2, 128, 128, 16, "mxfp8", "bf16")
    ws, yq, rope = c.space(4), torch.empty(c.T, 4, 128, device="cuda", dtype=torch.bfloat16), jfa.jfa_rope(128)
    call = lambda: jfa.jfa_rope_append(*c.args(), c.wq, c.wk, rope=rope, yq=yq, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1, 65, 16, 18, 190], [0, 70, 1, 17, 33]):
        c.x.normal_()
        c.lens.copy_(torch.tensor(lens))
        g.replay()
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        k, y = c.cache.k.clone(), yq.clone()
        for x in (c.cache.k, c.cache.v):
            x.fill_(119)
        want, _ = jfa.jfa_rope_append(*c.args(), c.wq, c.wk, rope=rope)
        for b, n in enumerate(lens):
            if n > 0:
                p, r = c.table_h[b, (n - 1) // 16], (n - 1) % 16
                assert torch.equal(k[p, :, r], c.cache.k[p, :, r])
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "mxfp8"), ("f32", "f32")])
def test_errors_found_on_the_device(dtype, cache):
    for dqk in (64, 32 + 8 if cache != "mxfp8" else 96):
        c = Case([2, 3], [20, 30], 2, 2, dqk, 64, 16, cache, dtype)
        ws, rope = c.space(2), jfa.jfa_rope(dqk)
        run = lambda **kw: jfa.jfa_rope_append(c.q, c.k, c.v, c.cache, kw.get("table", c.table), kw.get("offs", c.offs),
                                               kw.get("lens", c.lens), rope=rope, ws=ws)
        t = c.table.clone()
        t[1, 1] = c.pages
        before = c.cache.k.clone()
        run(table=t)
        assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
        rows = torch.ones(c.pages, 16, dtype=torch.bool, device="cuda")
        rows[c.table_h[0, 1], 2:4] = False  # sequence 0's two tokens, at 18 and 19: the others' page is bad
        m = rows[:, None, :, None].expand(before.shape)
        assert torch.equal(before[m], c.cache.k[m])
        for bad in (dict(offs=torch.tensor([0, 3, 4], device="cuda")), dict(offs=torch.tensor([1, 2, 5], device="cuda")),
                    dict(lens=torch.tensor([20, 10 ** 9], device="cuda")), dict(lens=torch.tensor([-1, 30], device="cuda"))):
            run(**bad)
            assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
        run()
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK


def test_no_tokens():
    c = Case([0, 0], [3, 0], 2, 2, 64, 64, 16, "bf16", "bf16")
    ws = c.space(2)
    yq, _ = jfa.jfa_rope_append(*c.args(), rope=jfa.jfa_rope(64), ws=ws)
    assert yq.shape == (0, 2, 64) and jfa.jfa_status_check(ws) == jfa.JFA_OK
    jfa.jfa_rope_append(c.q, c.k, c.v, c.cache, c.table, c.offs, torch.tensor([3, -1], device="cuda"), ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS


def test_refusals():
    c = Case([2], [2], 2, 2, 64, 64, 16, "bf16", "bf16")
    q, k, v, cache, t, o, n = c.args()
    for a in ((q[:, :, :32], k, v), (q, k[:, :1], v), (q, k, v[:1]), (q.float(), k, v), (q.transpose(1, 2), k, v), (q, k.cpu(), v)):
        with pytest.raises((ValueError, jfa.JfaError)):
            jfa.jfa_rope_append(*a, cache, t, o, n)
    for kw in (dict(wq=c.wq[:3]), dict(wk=c.wk.double()), dict(norm=False, wk=c.wk), dict(pos=torch.zeros(1, device="cuda").long()),
               dict(pos=torch.zeros(2, device="cuda")), dict(yq=torch.empty(2, 2, 32, device="cuda").bfloat16()), dict(planned=True)):
        with pytest.raises(ValueError):
            jfa.jfa_rope_append(q, k, v, cache, t, o, n, **kw)
    with pytest.raises(ValueError):
        jfa.jfa_rope_append(None, k, v, cache, t, o, n, yq=q)
    with pytest.raises(jfa.JfaError):
        jfa.jfa_rope_append(q, k, v, cache, t, o, n, rope=jfa.jfa_rope(66))


@pytest.mark.parametrize("mxfp8", [False, True])
def test_a_run_of_prompts_steps_and_candidates(mxfp8):
    """Prompts and then a token of each user, appended and attended under a window; then candidates behind
    each user's history.  The cache's own rows, read back, are the oracle's keys and values."""
    hq, hk, d, page, window, sinks = 4, 2, 64, 16, 30, 2
    cache = jfa.paged_cache(40, hk, d, page_size=page, mxfp8=mxfp8)
    order = torch.randperm(40, device="cuda").int()
    table = order[:16].reshape(2, 8).contiguous()
    rope, w = jfa.jfa_rope(d), torch.rand(d, device="cuda") + 0.5
    new_rows = lambda n: (torch.randn(n, h, d, device="cuda").bfloat16() for h in (hq, hk, hk))
    read = lambda t, n: [f64(x).transpose(1, 0, 2) for x in jfa.jfa_cache_read(
        cache, t[None].contiguous(), torch.tensor([0, n], device="cuda"), torch.tensor([n], device="cuda"), n)]
    lens = [0, 0]
    for new in ([40, 70], [1, 1], [1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        offs, lens_d = torch.tensor([0, new[0], sum(new)], device="cuda"), torch.tensor(lens, device="cuda")
        q, k, v = new_rows(sum(new))
        ws = jfa.jfa_paged_window_plan(q, cache, table, offs, lens_d, window, sinks=sinks)
        q, _ = jfa.jfa_rope_append(q, k, v, cache, table, offs, lens_d, w, w, rope=rope, ws=ws, planned=True)
        o, lse = jfa.jfa_paged_window_fwd(q, cache, table, offs, lens_d, window, sinks=sinks, ws=ws, planned=True)
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        seqs = [(int(offs[b]), *read(table[b], m), wref.window_mask(np.arange(m - n, m), np.arange(m), window, sinks))
                for b, (n, m) in enumerate(zip(new, lens))]
        wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 2, d ** -0.5, d), d, 100, "bf16")
    # three candidates of two tokens for each user, in pages of their own, at the positions behind the history
    own = order[16:22].reshape(6, 1).contiguous()
    offs, own_lens = torch.arange(0, 13, 2, device="cuda"), torch.full((6,), 2, device="cuda")
    pos = torch.cat([torch.arange(lens[b // 3], lens[b // 3] + 2) for b in range(6)]).cuda()
    q, k, v = new_rows(12)
    q, _ = jfa.jfa_rope_append(q, k, v, cache, own, offs, own_lens, w, w, rope=rope, pos=pos)
    o, lse = jfa.jfa_shared_fwd(q, cache, own, offs, own_lens, table, torch.tensor(lens, device="cuda"),
                                torch.tensor([0, 3, 6], device="cuda"))
    seqs = []
    for b in range(6):
        (pk, pv), (ok, ov) = read(table[b // 3], lens[b // 3]), read(own[b], 2)
        see = np.concatenate([np.ones((2, lens[b // 3]), bool), np.tri(2, dtype=bool)], 1)
        seqs.append((2 * b, np.concatenate([pk, ok], 1), np.concatenate([pv, ov], 1), see))
    wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 2, d ** -0.5, d), d, 100, "bf16")
