"""Attention behind shared prefixes (jfa_shared_fwd) against a plain 64-bit implementation.  What no
sequence owns is poisoned.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import window_ref as wref
from test_paged_gpu import DT, Batch, f64

pytestmark = pytest.mark.gpu


class Shared(Batch):
    """Sequences in groups: the prefixes are sequences of the same cache, without new tokens."""

    def __init__(self, groups, prefix, new, lens, hk, dqk, dv, page, cache, dtype, seed=0, wide=False):
        super().__init__(list(new) + [0] * len(prefix), list(lens) + list(prefix), hk, dqk, dv, page, cache, dtype, seed)
        self.G, self.S = len(groups), len(new)
        assert sum(groups) == self.S and len(prefix) == self.G
        self.group_h = np.concatenate([[0], np.cumsum(groups)]).astype(np.int64)
        self.groups = torch.tensor(self.group_h, device="cuda")
        self.prefix_table, self.prefix_lens = self.table[self.S:].contiguous(), self.lens[self.S:].clone()
        # a table of one page of 16 takes the kernel for few keys alone, a wider one the tiled kernels too
        width = self.table.shape[1] if wide else max([-(-int(n) // page) for n in lens] + [1])
        if wide and width * page <= 16:
            width = 2
        own = torch.nn.functional.pad(self.table[:self.S], (0, max(0, width - self.table.shape[1])), value=-1)
        self.own = (self.cache, own[:, :width].contiguous(), self.offs[:self.S + 1].clone(), self.lens[:self.S].clone())

    def call(self, q, **kw):
        return jfa.jfa_shared_fwd(q, *self.own, self.prefix_table, self.prefix_lens, self.groups, **kw)

    def want(self, q, hq, causal=True, scale=None):
        s = float(np.float32(self.dqk ** -0.5 if scale is None else scale))
        seqs = []
        for g in range(self.G):
            pk, pv, P = self.k_of(self.S + g), self.v_of(self.S + g), int(self.lens_h[self.S + g])
            for b in range(self.group_h[g], self.group_h[g + 1]):
                n, m = int(self.new[b]), int(self.lens_h[b])
                own = np.arange(m)[None] <= np.arange(m - n, m)[:, None] if causal else np.ones((n, m), bool)
                see = np.concatenate([np.ones((n, P), bool), own], 1)
                seqs.append((int(self.offs_h[b]), np.concatenate([pk, self.k_of(b)], 1),
                             np.concatenate([pv, self.v_of(b)], 1), see))
        return wref.attend(f64(q), seqs, hq // self.hk, s, self.dv)

    def longest(self):
        return int(self.lens_h[:self.S].max(initial=1)) + int(self.lens_h[self.S:].max(initial=1))


def space(b, hq):
    p = jfa.paged_params(*b.own, b.T, DT[b.dtype], heads_q=hq)
    return jfa.shared_workspace(p, b.G, b.prefix_table.shape[1])


def queries(b, hq, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(b.T, hq, b.dqk, generator=g, device="cuda").to(DT[b.dtype])


def check(b, hq, causal=True, q=None, scale=None, **kw):
    q = queries(b, hq) if q is None else q
    o, lse = b.call(q, causal=causal, scale=scale, **kw)
    wref.compare(f64(o), f64(lse), b.want(q, hq, causal, scale), b.dqk, b.longest(), b.dtype)
    return q, o, lse


def shape(kind):
    """(sequences of the groups, prefix lengths, new tokens, own lengths)."""
    rng = np.random.default_rng(3)
    if kind == "candidates":  # single tokens, cached just before
        g = [8, 1, 30]
        return g, [700, 33, 129], [1] * 39, [1] * 39
    if kind == "uncached":  # queries that see the prefix alone; a prefix without positions
        g = [5, 3, 7]
        return g, [300, 0, 64], rng.integers(1, 4, 15).tolist(), [0] * 15
    if kind == "continuations":
        g = [20]
        new = rng.integers(1, 3, 20)
        return g, [1000], new.tolist(), (new + rng.integers(0, 400, 20)).tolist()
    if kind == "ragged":  # empty groups, empty sequences, no prefix, no own keys, more tokens than keys
        g = [0, 4, 0, 3, 2, 6, 0]
        new = [0, 5, 1, 130, 64, 0, 33, 2, 70, 0, 0, 1, 17, 3, 300]
        lens = [0, 5, 0, 400, 64, 90, 20, 2, 71, 0, 5, 128, 17, 1, 900]
        return g, [50, 17, 0, 0, 513, 255, 64], new, lens
    if kind == "chunks":
        g = [3, 2]
        return g, [900, 130], [200, 150, 260, 300, 1], [200, 350, 260, 310, 64]
    if kind == "many":  # more than one CTA scans by itself: a launch of its own for the plan
        g = [40, 0, 660]
        return g, [100, 5, 333], [1] * 700, rng.integers(1, 30, 700).tolist()
    if kind in ("few keys", "few and more"):  # more sequences than a CTA checks
        g = [100, 1300, 3]
        new = rng.integers(0, 4, 1403)
        most = 16 if kind == "few keys" else 40
        return g, [70, 40, 200], new.tolist(), np.minimum(new + rng.integers(-1, most, 1403), most).clip(0).tolist()
    if kind == "few or many":  # by turns at the kernel for few's bound
        n = 60
        own = np.array([16, 17, 0, 200, 15, 16])[np.arange(n) % 6]
        return [n // 2, n // 2], [300, 77], (1 + np.arange(n) % 3).tolist(), own.tolist()
    if kind == "many groups":
        g = rng.integers(0, 3, 600).tolist()
        n = sum(g)
        return g, rng.integers(0, 40, 600).tolist(), [1] * n, rng.integers(0, 5, n).tolist()
    raise KeyError(kind)


CASES = [
    # kind, dtype, cache, hq, hk, dqk, dv, page, causal
    ("candidates", "f32", "f32", 4, 2, 64, 64, 16, True),
    ("ragged", "f32", "f32", 3, 1, 40, 24, 32, True),
    ("ragged", "f32", "mxfp8", 2, 2, 32, 96, 16, False),
    ("ragged", "bf16", "bf16", 4, 2, 72, 8, 16, True),
    ("candidates", "bf16", "bf16", 8, 8, 64, 64, 16, True),
    ("candidates", "bf16", "bf16", 8, 2, 128, 128, 64, True),
    ("candidates", "bf16", "mxfp8", 32, 4, 128, 128, 32, True),
    ("uncached", "bf16", "bf16", 8, 2, 128, 64, 64, True),
    ("uncached", "bf16", "mxfp8", 3, 1, 64, 128, 128, True),
    ("uncached", "f32", "f32", 2, 2, 64, 64, 16, False),
    ("continuations", "bf16", "bf16", 8, 1, 128, 128, 64, True),
    ("continuations", "bf16", "mxfp8", 16, 4, 128, 128, 64, True),
    ("continuations", "bf16", "mxfp8", 4, 4, 64, 64, 16, False),
    ("ragged", "bf16", "bf16", 4, 4, 128, 128, 64, True),
    ("ragged", "bf16", "bf16", 8, 1, 64, 64, 16, False),
    ("ragged", "bf16", "mxfp8", 9, 3, 64, 128, 64, True),
    ("ragged", "bf16", "mxfp8", 4, 1, 128, 128, 32, True),
    ("ragged", "bf16", "bf16", 20, 1, 64, 128, 256, True),
    ("chunks", "bf16", "bf16", 8, 2, 128, 128, 128, True),
    ("chunks", "bf16", "mxfp8", 4, 2, 128, 64, 64, True),
    ("chunks", "bf16", "bf16", 130, 1, 64, 64, 64, True),
    ("many", "bf16", "bf16", 4, 4, 64, 64, 16, True),
    ("many", "bf16", "mxfp8", 8, 2, 128, 128, 16, True),
    ("few and more", "bf16", "bf16", 8, 2, 128, 128, 16, True),
    ("few or many", "bf16", "mxfp8", 8, 2, 64, 64, 16, True),
    ("few or many", "bf16", "bf16", 8, 1, 128, 64, 64, True),
    ("few or many", "f32", "f32", 3, 3, 40, 48, 32, False),
    ("few keys", "bf16", "bf16", 6, 1, 64, 64, 16, True),
    ("few keys", "bf16", "mxfp8", 2, 2, 128, 96, 16, True),
    ("few keys", "bf16", "bf16", 2, 1, 40, 24, 16, False),
    ("few keys", "f32", "f32", 4, 4, 64, 128, 16, True),
    ("few keys", "f32", "mxfp8", 5, 1, 32, 64, 16, False),
    ("many groups", "bf16", "bf16", 8, 2, 64, 64, 16, True),
    ("many groups", "f32", "f32", 2, 1, 32, 32, 16, True),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", CASES, ids=["%s-%s-%s-%d-%d-D%d-%d-p%d-%d" % c for c in CASES])
def test_attention(case, wide):
    kind, dtype, cache, hq, hk, dqk, dv, page, causal = case
    b = Shared(*shape(kind), hk, dqk, dv, page, cache, dtype, wide=wide)
    ws = space(b, hq)
    q, o, lse = check(b, hq, causal, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    o2, lse2 = b.call(q, causal=causal, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_scores_of_any_size_meet():
    """Rows whose prefix outweighs their own keys by far, and the other way round."""
    b = Shared([6], [100], [1] * 6, [20] * 6, 2, 64, 64, 16, "bf16", "bf16")
    for s in (30.0, 0.001):
        check(b, 8, scale=s)


def test_strides_streams_and_given_outputs():
    b = Shared(*shape("ragged"), 2, 64, 64, 16, "bf16", "bf16")
    q = torch.randn(b.T, 12, 64, device="cuda").bfloat16()[:, 4:8]
    o, lse = torch.empty(b.T, 4, 64, device="cuda", dtype=torch.bfloat16), torch.empty(b.T, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = b.call(q, o=o, lse=lse, stream=s)
    s.synchronize()
    assert o2 is o and lse2 is lse
    wref.compare(f64(o), f64(lse), b.want(q, 4), 64, b.longest(), "bf16")


def test_captured_and_replayed():
    """A captured call serves other lengths, prefixes and groups of as many sequences."""
    b = Shared([4, 4], [500, 300], [1] * 8, [40] * 8, 2, 128, 128, 64, "bf16", "bf16")
    q, ws = queries(b, 8), space(b, 8)
    o, lse = torch.empty(b.T, 8, 128, device="cuda", dtype=torch.bfloat16), torch.empty(b.T, 8, device="cuda")
    call = lambda: b.call(q, o=o, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for groups, prefix, lens in (([0, 4, 8], [500, 300], [40] * 8), ([0, 1, 8], [33, 299], [0, 3, 40, 1, 1, 7, 30, 0]),
                                 ([0, 8, 8], [0, 300], [5] * 8)):
        b.group_h = np.array(groups, np.int64)
        b.lens_h = np.array(lens + prefix, np.int64)
        b.groups.copy_(torch.tensor(groups))
        b.own[3].copy_(torch.tensor(lens))
        b.prefix_lens.copy_(torch.tensor(prefix))
        q.normal_()
        g.replay()
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        wref.compare(f64(o), f64(lse), b.want(q, 8), 128, 600, "bf16")


def spoiled(t, at, value):
    t = t.clone()
    t[at] = value
    return t


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [3, 300, 600])
def test_errors_found_on_the_device(n, wide):
    """Invalid groups, prefixes and sequences leave the outputs alone; bad pages read as zeros."""
    b = Shared([n, n], [100, 200], [1] * 2 * n, [5] * 2 * n, 2, 64, 64, 16, "bf16", "bf16", wide=wide)
    q, ws = queries(b, 4), space(b, 4)
    good = (b.own[1], b.own[2], b.own[3], b.prefix_table, b.prefix_lens, b.groups)
    o, lse = torch.full((b.T, 4, 64), 7.0, device="cuda").bfloat16(), torch.full((b.T, 4), 7.0, device="cuda")
    for i, at, value in ((5, 0, 1), (5, 1, 2 * n + 1), (5, 1, -1), (5, 2, 2 * n - 1), (4, 0, -1), (4, 1, 10 ** 9),
                         (1, 1, -5), (1, 2 * n, 0), (2, 1, -1), (2, 0, 10 ** 9)):
        x = list(good)
        x[i] = spoiled(x[i], at, value)
        jfa.jfa_shared_fwd(q, b.cache, *x, o=o, lse=lse, ws=ws)
        assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS, (i, at, value)
        assert bool((o == 7).all()) and bool((lse == 7).all())
    for i in (0, 3):
        x = list(good)
        x[i] = spoiled(x[i], (0, 0), -7)
        jfa.jfa_shared_fwd(q, b.cache, *x, ws=ws)
        assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
    jfa.jfa_shared_fwd(q, b.cache, *good, o=o, lse=lse, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    wref.compare(f64(o), f64(lse), b.want(q, 4), 64, b.longest(), "bf16")


@pytest.mark.parametrize("kind,cache", [("few", "bf16"), ("few", "mxfp8"), ("many", "bf16"), ("many", "mxfp8")])
def test_a_wait_that_runs_out(kind, cache):
    b = (Shared([2], [9000], [1, 1], [5, 5], 2, 128, 128, 64, cache, "bf16") if kind == "few" else
         Shared([2], [3000], [200, 300], [200, 300], 2, 128, 128, 64, cache, "bf16"))
    q, ws = queries(b, 8), space(b, 8)
    jfa.jfa_test_hold(True)
    try:
        b.call(q, ws=ws)
        st = jfa.jfa_status_check(ws)
    finally:
        jfa.jfa_test_hold(False)
    assert st == jfa.JFA_ERR_TIMEOUT
    check(b, 8, q=q, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK


def test_empty_calls():
    b = Shared([2], [50], [0, 0], [5, 0], 2, 64, 64, 16, "bf16", "bf16")
    ws = space(b, 2)
    o, lse = b.call(queries(b, 2), ws=ws)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2) and jfa.jfa_status_check(ws) == jfa.JFA_OK
    e = lambda *n, t=torch.int64: torch.zeros(n, dtype=t, device="cuda")
    jfa.jfa_shared_fwd(queries(b, 2), b.cache, e(0, 3, t=torch.int32), e(1), e(0), e(0, 2, t=torch.int32), e(0), e(1), ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK


def test_refusals():
    b = Shared([2], [50], [1, 1], [5, 5], 2, 64, 64, 16, "bf16", "bf16")
    q = queries(b, 2)
    c, t, f, n = b.own
    bad = [dict(groups=b.groups.int()), dict(groups=b.groups[:1]), dict(prefix_lens=b.prefix_lens.cpu()),
           dict(prefix_table=b.prefix_table.long()), dict(prefix_table=b.prefix_table[0]), dict(groups=b.groups[None])]
    for kw in bad:
        x = dict(prefix_table=b.prefix_table, prefix_lens=b.prefix_lens, groups=b.groups)
        x.update(kw)
        with pytest.raises(ValueError):
            jfa.jfa_shared_fwd(q, c, t, f, n, x["prefix_table"], x["prefix_lens"], x["groups"])
    with pytest.raises(jfa.JfaError) as e:
        b.call(q, ws=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.code == jfa.JFA_ERR_WORKSPACE
    empty = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(jfa.JfaError) as e:  # sequences, but no group
        jfa.jfa_shared_fwd(q, c, t, f, n, empty, torch.zeros(0, dtype=torch.int64, device="cuda"), b.groups[:1])
    assert e.value.code == jfa.JFA_ERR_INVALID_ARG
