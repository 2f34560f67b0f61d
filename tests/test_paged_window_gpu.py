"""Attention over a window of a paged cache with sinks (jfa_paged_window_plan, jfa_paged_window_fwd)
against a plain 64-bit implementation.  What no query sees, and the pages that hold nothing else, are
poisoned throughout.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref
import window_ref as wref
from test_paged_gpu import DT, EDGES, Batch, f64, ragged

pytestmark = pytest.mark.gpu


def want(b, q, hq, window, sinks, scale=None):
    s = float(np.float32(b.dqk ** -0.5 if scale is None else scale))
    seqs = []
    for x in range(b.B):
        n, m = int(b.new[x]), int(b.lens_h[x])
        see = wref.window_mask(np.arange(m - n, m), np.arange(m), window, sinks)
        seqs.append((int(b.offs_h[x]), b.k_of(x), b.v_of(x), see))
    return wref.attend(f64(q), seqs, hq // b.hk, s, b.dv)


def queries(b, hq, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(b.T, hq, b.dqk, generator=g, device="cuda").to(DT[b.dtype])


def check(b, hq, window, sinks, q=None, poison=True, scale=None, **kw):
    q = queries(b, hq) if q is None else q
    if poison:
        wref.poison_hidden(b, window, sinks)
    o, lse = jfa.jfa_paged_window_fwd(q, *b.args(), window, sinks=sinks, scale=scale, **kw)
    wref.compare(f64(o), f64(lse), want(b, q, hq, window, sinks, scale), b.dqk, int(b.lens_h.max(initial=1)), b.dtype)
    return q, o, lse


def space(b, hq):
    return jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, DT[b.dtype], heads_q=hq))


CASES = [
    # kind, dtype, cache, hq, hk, dqk, dv, page, window, sinks
    ("step", "f32", "f32", 4, 2, 64, 64, 16, 1, 0),
    ("step", "f32", "mxfp8", 4, 2, 64, 32, 32, 100, 4),
    ("chunk", "f32", "f32", 3, 1, 40, 24, 32, 33, 2),
    ("prompt", "f32", "f32", 2, 2, 128, 128, 64, 64, 0),
    ("chunk", "bf16", "bf16", 4, 2, 72, 8, 16, 50, 17),
    ("step", "bf16", "bf16", 8, 8, 64, 64, 16, 1, 1),
    ("step", "bf16", "bf16", 8, 1, 128, 128, 64, 128, 4),
    ("step", "bf16", "bf16", 8, 1, 128, 128, 64, 65, 0),
    ("step", "bf16", "mxfp8", 32, 4, 128, 128, 32, 77, 5),
    ("step", "bf16", "mxfp8", 3, 1, 64, 64, 128, 200, 1),
    ("step", "bf16", "mxfp8", 16, 1, 128, 64, 16, 31, 33),
    ("step", "bf16", "bf16", 20, 1, 64, 128, 256, 90, 64),
    ("chunk", "bf16", "bf16", 4, 4, 128, 128, 64, 1, 0),
    ("chunk", "bf16", "bf16", 4, 4, 128, 128, 64, 100, 3),
    ("chunk", "bf16", "bf16", 8, 1, 64, 64, 16, 129, 130),
    ("chunk", "bf16", "mxfp8", 4, 1, 128, 128, 32, 60, 4),
    ("chunk", "bf16", "mxfp8", 9, 3, 64, 128, 64, 300, 0),
    ("chunk", "bf16", "mxfp8", 40, 1, 128, 128, 16, 20, 20),
    ("prompt", "bf16", "bf16", 2, 2, 128, 128, 128, 128, 1),
    ("prompt", "bf16", "bf16", 8, 1, 64, 64, 256, 17, 0),
    ("prompt", "bf16", "bf16", 4, 2, 128, 64, 32, 5000, 9),
    ("prompt", "bf16", "mxfp8", 6, 2, 128, 128, 64, 250, 140),
    ("one long", "bf16", "bf16", 8, 1, 128, 128, 64, 1000, 4),
    ("one long", "bf16", "mxfp8", 4, 2, 64, 64, 32, 3000, 0),
    ("one long chunk", "bf16", "bf16", 8, 2, 128, 128, 64, 400, 4),
    ("one long chunk", "bf16", "mxfp8", 8, 1, 128, 128, 16, 1500, 300),
    ("many short", "bf16", "bf16", 4, 4, 64, 64, 16, 7, 2),
    ("many short", "bf16", "mxfp8", 8, 2, 128, 128, 16, 20, 0),
    ("mixed", "bf16", "bf16", 8, 2, 128, 128, 64, 96, 4),
    ("chunk", "bf16", "bf16", 130, 1, 64, 64, 64, 30, 4),
]


@pytest.mark.parametrize("case", CASES, ids=["%s-%s-%s-%d-%d-D%d-%d-p%d-w%d-s%d" % c for c in CASES])
def test_attention(case):
    kind, dtype, cache, hq, hk, dqk, dv, page, window, sinks = case
    b = Batch(*ragged(kind), hk, dqk, dv, page, cache, dtype)
    ws = space(b, hq)
    q, o, lse = check(b, hq, window, sinks, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    # and on a plan, bit for bit
    jfa.jfa_paged_window_plan(q, *b.args(), window, sinks=sinks, ws=ws)
    o2, lse2 = jfa.jfa_paged_window_fwd(q, *b.args(), window, sinks=sinks, ws=ws, planned=True)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    if b.B <= 512:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    else:
        wref.compare(f64(o2), f64(lse2), want(b, q, hq, window, sinks), dqk, int(b.lens_h.max()), dtype)


@pytest.mark.parametrize("cache", ["bf16", "mxfp8"])
@pytest.mark.parametrize("kind", ["step", "chunk"])
def test_a_window_of_everything_is_plain_attention(kind, cache):
    b = Batch(*ragged(kind), 2, 128, 128, 64, cache, "bf16")
    q = queries(b, 8)
    o, lse = jfa.jfa_paged_fwd(q, *b.args())
    most = int(b.lens_h.max())  # a window, or sinks, of as many keys show all of them
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 40, 2 ** 40), (most, 0), (1, most)):
        o2, lse2 = jfa.jfa_paged_window_fwd(q, *b.args(), window, sinks=sinks)
        assert torch.equal(torch.isfinite(lse), torch.isfinite(lse2))
        fin = torch.isfinite(lse)
        # the work is cut elsewhere, so that sums meet in another order: fp32 sums, one rounding to bf16
        assert torch.allclose(lse[fin], lse2[fin], rtol=0, atol=2e-5)
        assert float((o.float() - o2.float()).norm() / o.float().norm()) < 2.0 ** -8


def test_window_of_one_key_is_its_value():
    b = Batch([3, 1, 40], [40, 17, 40], 2, 64, 64, 16, "bf16", "bf16")
    wref.poison_hidden(b, 1, 0)
    _, o, lse = check(b, 2, 1, 0, poison=False)
    for x in range(b.B):
        n, m = int(b.new[x]), int(b.lens_h[x])
        v = b.v_of(x)[:, m - n:].transpose(1, 0, 2)
        assert np.array_equal(f64(o)[b.offs_h[x]:b.offs_h[x + 1]], v)


def test_strides_streams_and_given_outputs():
    b = Batch(*ragged("chunk"), 2, 64, 64, 16, "bf16", "bf16")
    wide = torch.randn(b.T, 12, 64, device="cuda").bfloat16()
    q = wide[:, 4:8]
    o, lse = torch.empty(b.T, 4, 64, device="cuda", dtype=torch.bfloat16), torch.empty(b.T, 4, device="cuda")
    wref.poison_hidden(b, 40, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = jfa.jfa_paged_window_fwd(q, *b.args(), 40, sinks=4, o=o, lse=lse, stream=s)
    s.synchronize()
    assert o2 is o and lse2 is lse
    wref.compare(f64(o), f64(lse), want(b, q, 4, 40, 4), 64, 1100, "bf16")


def test_captured_and_replayed_with_longer_caches():
    """A captured step serves later lengths and other pages."""
    b = Batch([1] * 4, [40, 200, 64, 500], 2, 128, 128, 64, "bf16", "bf16")
    q, ws = queries(b, 8), space(b, 8)
    o, lse = torch.empty(b.T, 8, 128, device="cuda", dtype=torch.bfloat16), torch.empty(b.T, 8, device="cuda")
    call = lambda: jfa.jfa_paged_window_fwd(q, *b.args(), 100, sinks=4, o=o, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([40, 200, 64, 500], [39, 101, 1, 499], [3, 128, 63, 100]):
        b.lens_h = np.array(lens, np.int64)
        b.lens.copy_(torch.tensor(lens))
        q.normal_()
        g.replay()
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        wref.compare(f64(o), f64(lse), want(b, q, 8, 100, 4), 128, 500, "bf16")


def test_errors_found_on_the_device():
    for cache, hq in (("bf16", 4), ("mxfp8", 4)):
        for new, lens in (([1, 2], [300, 200]), ([200, 100], [300, 200])):
            b = Batch(new, lens, 2, 64, 64, 16, cache, "bf16")
            q, ws = queries(b, hq), space(b, hq)
            b.table[0, 10] = b.pages  # inside the window
            jfa.jfa_paged_window_fwd(q, *b.args(), 250, sinks=4, ws=ws)
            assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
            o = torch.full((b.T, hq, 64), 7.0, device="cuda", dtype=torch.bfloat16)
            lens_bad = b.lens.clone()
            lens_bad[1] = 10 ** 9
            jfa.jfa_paged_window_fwd(q, b.cache, b.table, b.offs, lens_bad, 50, sinks=4, o=o, ws=ws)
            assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
            assert bool((o == 7).all())


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("kind,cache,hq", [("few", "bf16", 8), ("few", "mxfp8", 32), ("many", "bf16", 8), ("many", "mxfp8", 8)])
def test_a_wait_that_runs_out(kind, cache, hq, planned):
    if kind == "few":
        b = Batch([1, 2, 1], [9000, 5000, 7000], 2, 128, 128, 64, cache, "bf16")
    else:
        b = Batch([700, 300], [900, 3000], 2, 128, 128, 64, cache, "bf16")
    q, ws = queries(b, hq), space(b, hq)
    plan = lambda: jfa.jfa_paged_window_plan(q, *b.args(), 600, sinks=4, ws=ws) if planned else None
    plan()
    jfa.jfa_test_hold(True)
    try:
        jfa.jfa_paged_window_fwd(q, *b.args(), 600, sinks=4, ws=ws, planned=planned)
        st = jfa.jfa_status_check(ws)
    finally:
        jfa.jfa_test_hold(False)
    assert st == jfa.JFA_ERR_TIMEOUT
    plan()
    check(b, hq, 600, 4, q=q, ws=ws, planned=planned)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK


def test_refusals():
    b = Batch([1, 1], [10, 10], 2, 64, 64, 16, "bf16", "bf16")
    q = queries(b, 2)
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(ValueError):
            jfa.jfa_paged_window_fwd(q, *b.args(), window, sinks=sinks)
        with pytest.raises(ValueError):
            jfa.jfa_paged_window_plan(q, *b.args(), window, sinks=sinks)
    with pytest.raises(ValueError):
        jfa.jfa_paged_window_fwd(q, *b.args(), 4, planned=True)
    with pytest.raises(ValueError):
        jfa.jfa_paged_window_fwd(q.cpu(), *b.args(), 4)
