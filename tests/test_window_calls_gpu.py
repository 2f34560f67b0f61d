"""Windows, shared prefixes and appending where calls meet: caches past 32 bits, calls at once on two streams,
prefixes that several groups share, plans that were made for another window.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import window_ref as wref
from test_paged_gpu import DT, Batch, f64, ragged
from test_paged_window_gpu import queries, space, want
from test_shared_gpu import Shared
from test_shared_gpu import space as shared_space
from test_window_gpu import batch, compare, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
def test_caches_past_32_bits(kind):
    """Pages whose elements lie past 2^32 (values and, in MXFP8, bytes): prompts appended there, then attended
    under a window and as prefixes."""
    pages, hk, hq, page, d = 70000, 8, 16, 64, 128
    if kind == "bf16":
        c = jfa.PagedCache(*(torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    else:
        u = lambda n: torch.empty(pages, hk, page, n, dtype=torch.uint8, device="cuda")
        c = jfa.PagedCache(u(d), u(d), u(d // 32), u(d // 32))
    assert c.k.numel() > 2 ** 32
    lens = [350, 230]
    at = np.cumsum([0] + lens)
    dev = lambda x: torch.tensor(x, device="cuda")
    table = (pages - 1 - torch.arange(12, device="cuda").int()).view(2, 6).contiguous()
    k, v = (torch.randn(sum(lens), hk, d, device="cuda").bfloat16() for _ in range(2))
    jfa.jfa_rope_append(None, k, v, c, table, dev(at), dev(lens), norm=False)
    kr, vr = jfa.jfa_cache_read(c, table, dev(at), dev(lens), sum(lens))
    if kind == "bf16":
        assert torch.equal(kr, k) and torch.equal(vr, v)
    part = lambda x, b: f64(x[at[b]:at[b + 1]]).transpose(1, 0, 2)
    scale = float(np.float32(d ** -0.5))
    for new in (1, 200):
        q = torch.randn(2 * new, hq, d, device="cuda").bfloat16()
        offs = dev([0, new, 2 * new])
        o, lse = jfa.jfa_paged_window_fwd(q, c, table, offs, dev(lens), 100, sinks=3)
        seqs = [(b * new, part(kr, b), part(vr, b), wref.window_mask(np.arange(n - new, n), np.arange(n), 100, 3))
                for b, n in enumerate(lens)]
        wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 2, scale, d), d, 350, "bf16")
        # the second sequence's first 9 positions behind the first's 350, and the other way round
        o, lse = jfa.jfa_shared_fwd(q, c, table.flip(0), offs, dev([9, 40]), table, dev(lens), dev([0, 1, 2]))
        seqs = []
        for b, n in enumerate((9, 40)):
            own = np.arange(n)[None] <= np.arange(n - new, n)[:, None]
            seqs.append((b * new, np.concatenate([part(kr, b), part(kr, 1 - b)[:, :n]], 1),
                         np.concatenate([part(vr, b), part(vr, 1 - b)[:, :n]], 1),
                         np.concatenate([np.ones((new, lens[b]), bool), own], 1)))
        wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 2, scale, d), d, 400, "bf16")


def test_calls_at_once():
    """Calls of two streams that run side by side, each with its workspace, give what they give alone."""
    def work(seed):
        b = Batch(*ragged("chunk"), 2, 128, 128, 64, "mxfp8", "bf16", seed=seed)
        s = Shared([30, 9], [700, 130], [1] * 39, [5, 40, 1] * 13, 2, 128, 128, 64, "bf16", "bf16", seed=seed)
        q, k, v, do, offs = batch([700, 0, 129, 1100], 4, 128, 128, "bf16", seed)
        pq, sq = queries(b, 8, seed), queries(s, 8, seed)

        def run(stream=None):
            out = list(jfa.jfa_paged_window_fwd(pq, *b.args(), 60, sinks=4, stream=stream))
            out += s.call(sq, stream=stream)
            o, lse = jfa.jfa_window_fwd(q, k, v, offs, 200, sinks=2, stream=stream)
            return out + [o, lse, *jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 200, sinks=2, stream=stream)]

        return run

    runs = [work(1), work(2)]
    alone = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = [r(s) for r, s in zip(runs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_prefixes_that_groups_share():
    """Two groups behind one prefix, and a sequence whose own pages are its prefix's."""
    b = Shared([3, 2], [200, 90], [2, 1, 30, 1, 3], [20, 9, 30, 90, 14], 2, 64, 64, 16, "bf16", "bf16")
    b.prefix_table[1], b.prefix_lens[1] = b.prefix_table[0], 200
    b.table_h[b.S + 1], b.lens_h[b.S + 1] = b.table_h[b.S], 200
    b.own[1][4] = b.prefix_table[0, :b.own[1].shape[1]]
    b.table_h[4, :b.own[1].shape[1]] = b.table_h[b.S, :b.own[1].shape[1]]
    q, ws = queries(b, 8), shared_space(b, 8)
    o, lse = b.call(q, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    # sequence 4's own keys are the first 14 of the prefix, group 1's prefix is group 0's
    k0, v0 = b.k_of(b.S), b.v_of(b.S)
    scale, seqs = float(np.float32(64 ** -0.5)), []
    for x in range(b.S):
        n, m = int(b.new[x]), int(b.lens_h[x])
        k, v = (k0[:, :m], v0[:, :m]) if x == 4 else (b.k_of(x), b.v_of(x))
        see = np.concatenate([np.ones((n, 200), bool), np.arange(m)[None] <= np.arange(m - n, m)[:, None]], 1)
        seqs.append((int(b.offs_h[x]), np.concatenate([k0, k], 1), np.concatenate([v0, v], 1), see))
    wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 4, scale, 64), 64, 300, "bf16")


def test_plans_of_another_window():
    """They give wrong results within the buffers' bounds; the next call is right again."""
    lens = [700, 3, 300]
    q, k, v, do, offs = batch(lens, 2, 128, 128, "bf16")
    T, pad = sum(lens), 64
    ws = jfa.workspace(jfa.params_for(q, k, v, offs, None, True))
    whole = [torch.full((T + 2 * pad, 2, 128), 7.0, device="cuda").bfloat16() for _ in range(4)]
    o, dq, dk, dv = (x[pad:-pad] for x in whole)
    lse = torch.empty(T, 2, device="cuda")
    for plan in (lambda: jfa.jfa_plan(q, k, v, offs, causal=True, ws=ws),
                 lambda: jfa.jfa_window_plan(q, k, v, offs, 1, ws=ws),
                 lambda: jfa.jfa_window_plan(q, k, v, offs, 600, sinks=300, ws=ws)):
        plan()
        jfa.jfa_window_fwd(q, k, v, offs, 200, sinks=4, o=o, lse=lse, ws=ws, planned=True)
        jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 200, sinks=4, dq=dq, dk=dk, dv=dv, ws=ws, planned=True)
        for x in whole:
            assert bool((x[:pad] == 7).all()) and bool((x[-pad:] == 7).all())
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, 200, sinks=4, ws=ws)
    g = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 200, sinks=4, ws=ws)
    compare(dict(zip(("o", "lse", "dq", "dk", "dv"), (f64(x) for x in (o, lse, *g)))),
            reference(*(f64(x) for x in (q, k, v, do)), lens, 200, 4, float(np.float32(128 ** -0.5))), "bf16")
    for kind, cache, hq in (("step", "bf16", 8), ("chunk", "bf16", 8), ("chunk", "mxfp8", 8)):
        b = Batch(*ragged(kind), 2, 128, 128, 64, cache, "bf16")
        pq, pws = queries(b, hq), space(b, hq)
        whole = torch.full((b.T + 2 * pad, hq, 128), 7.0, device="cuda").bfloat16()
        o, lse = whole[pad:-pad], torch.empty(b.T, hq, device="cuda")
        for plan in (lambda: jfa.jfa_paged_plan(pq, *b.args(), ws=pws),
                     lambda: jfa.jfa_paged_window_plan(pq, *b.args(), 1, ws=pws),
                     lambda: jfa.jfa_paged_window_plan(pq, *b.args(), 300, sinks=64, ws=pws)):
            plan()
            jfa.jfa_paged_window_fwd(pq, *b.args(), 77, sinks=2, o=o, lse=lse, ws=pws, planned=True)
            assert bool((whole[:pad] == 7).all()) and bool((whole[-pad:] == 7).all())
        o, lse = jfa.jfa_paged_window_fwd(pq, *b.args(), 77, sinks=2, ws=pws)
        wref.compare(f64(o), f64(lse), want(b, pq, hq, 77, 2), 128, int(b.lens_h.max()), "bf16")


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "mxfp8"), ("f32", "f32")])
@pytest.mark.parametrize("new", [1, 3, 200])
def test_the_longest_cache(dtype, cache, new):
    """The last positions of a cache as long as calls allow: tokens appended there, and attended under a window
    whose pages alone are in the table."""
    page, hk, hq, d, window, sinks = 256, 2, 8, 64, 100, 5
    width = (2 ** 31 - 256) // page
    n = width * page  # 2^31 - 256
    c = jfa.paged_cache(5, hk, d, page_size=page, dtype=DT[dtype], mxfp8=cache == "mxfp8")
    dev = lambda x: torch.tensor(x, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(new)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -2], table[0, -1] = 3, 0, 4
    # the first page and the last two as a sequence of their own, filled; then the new tokens over its end
    short = table[:, [0, -2, -1]].contiguous()
    m = 3 * page
    jfa.jfa_cache_write(r(m, hk, d), r(m, hk, d), c, short, dev([0, m]), dev([m]))
    q, k, v = r(new, hq, d), r(new, hk, d), r(new, hk, d)
    ws = jfa.paged_workspace(jfa.paged_params(c, table, dev([0, new]), dev([n]), new, DT[dtype], heads_q=hq))
    q, _ = jfa.jfa_rope_append(q, k, v, c, table, dev([0, new]), dev([n]), norm=False, rope=jfa.jfa_rope(d), ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    kr, vr = jfa.jfa_cache_read(c, short, dev([0, m]), dev([m]), m, dtype=DT[dtype])
    assert torch.equal(vr[m - new:], v) or cache == "mxfp8"
    at = np.concatenate([np.arange(page), np.arange(n - 2 * page, n)])
    see = wref.window_mask(np.arange(n - new, n), at, window, sinks)
    want = wref.attend(f64(q), [(0, f64(kr).transpose(1, 0, 2), f64(vr).transpose(1, 0, 2), see)], hq // hk,
                       float(np.float32(d ** -0.5)), d)
    for planned in (False, True):
        if planned:
            jfa.jfa_paged_window_plan(q, c, table, dev([0, new]), dev([n]), window, sinks=sinks, ws=ws)
        o, lse = jfa.jfa_paged_window_fwd(q, c, table, dev([0, new]), dev([n]), window, sinks=sinks, ws=ws, planned=planned)
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        wref.compare(f64(o), f64(lse), want, d, m, dtype)


def test_tables_without_pages():
    """Groups without prefixes, sequences without keys of their own, and neither."""
    b = Shared([2, 3], [70, 33], [1, 2, 1, 20, 3], [5, 9, 1, 20, 40], 2, 64, 64, 16, "bf16", "bf16")
    q = queries(b, 4)
    c, table, offs, lens = b.own
    none = lambda n: torch.empty(n, 0, dtype=torch.int32, device="cuda")
    zeros = lambda n: torch.zeros(n, dtype=torch.int64, device="cuda")
    o, lse = jfa.jfa_shared_fwd(q, c, table, offs, lens, none(2), zeros(2), b.groups)
    o2, lse2 = jfa.jfa_paged_fwd(q, c, table, offs, lens)
    assert float((o.float() - o2.float()).abs().max()) <= 2.0 ** -5 and torch.allclose(lse, lse2, atol=1e-5)
    o, lse = jfa.jfa_shared_fwd(q, c, none(5), offs, zeros(5), b.prefix_table, b.prefix_lens, b.groups)
    scale, seqs = float(np.float32(64 ** -0.5)), []
    for x in range(5):
        g = int(x >= 2)
        n, m = int(b.new[x]), int(b.lens_h[b.S + g])
        seqs.append((int(b.offs_h[x]), b.k_of(b.S + g), b.v_of(b.S + g), np.ones((n, m), bool)))
    wref.compare(f64(o), f64(lse), wref.attend(f64(q), seqs, 2, scale, 64), 64, 100, "bf16")
    o, lse = jfa.jfa_shared_fwd(q, c, none(5), offs, zeros(5), none(2), zeros(2), b.groups)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    # a window over sequences without pages
    o, lse = jfa.jfa_paged_window_fwd(q, c, none(5), offs, zeros(5), 7, sinks=1)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
