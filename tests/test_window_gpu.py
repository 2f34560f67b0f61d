"""Causal attention over a sliding window with sinks on jagged tensors (jfa_window_plan, _fwd, _bwd) against a
plain 64-bit implementation, its gradients also against differences.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import parity_util as pu
import window_ref as wref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
f64 = pu.to64


def batch(lens, H, dqk, dv, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = int(sum(lens))
    q, k, v, do = (torch.randn(T, H, d, generator=g, device="cuda").to(DT[dtype]) for d in (dqk, dqk, dv, dv))
    offs = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device="cuda")
    return q, k, v, do, offs


def reference(q, k, v, do, lens, window, sinks, scale):
    """o, lse and the gradients, a head of a sequence at a time, from the formulas."""
    out = {n: np.zeros(x.shape) for n, x in (("o", v), ("dq", q), ("dk", k), ("dv", v))}
    out["lse"] = np.zeros(q.shape[:2])
    out["size"] = {n: np.zeros(out[n].shape) for n in ("o", "dq", "dk", "dv")}
    out["rel"] = 0.0
    t = 0
    for n in lens:
        i = np.arange(n)
        see = wref.window_mask(i, i, window, sinks)
        for h in range(q.shape[1]):
            a, b, c, d = (x[t:t + n, h] for x in (q, k, v, do))
            if n == 0:
                continue
            s = np.where(see, scale * (a @ b.T), -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p /= l
            o = p @ c
            ds = p * (d @ c.T - np.sum(d * o, 1, keepdims=True))
            out["o"][t:t + n, h], out["lse"][t:t + n, h] = o, (m + np.log(l))[:, 0]
            out["dq"][t:t + n, h], out["dk"][t:t + n, h], out["dv"][t:t + n, h] = scale * ds @ b, scale * ds.T @ a, p.T @ d
            # what the sums are of, and the relative error that fp32 leaves (below)
            w = p * (np.abs(d) @ np.abs(c).T + np.sum(np.abs(d * o), 1, keepdims=True))
            for name, x in (("o", p @ np.abs(c)), ("dq", scale * w @ np.abs(b)), ("dk", scale * w.T @ np.abs(a)),
                            ("dv", p.T @ np.abs(d))):
                out["size"][name][t:t + n, h] = x
            mag = scale * np.max(np.abs(a) @ np.abs(b).T)
            out["rel"] = max(out["rel"], 2.0 ** -23 * (q.shape[2] + v.shape[2] + n + 32 + mag * (q.shape[2] + 8)))
        t += n
    return out


def compare(got, want, dtype):
    """bf16: the bounds of the other jagged kernels.  fp32: a weight is off by its score's error (dim products of
    at most `mag` in all, each step within 2^-23, and exp2), a sum over n terms by n such steps; an element is
    within the sum of these times what it is the sum of."""
    if dtype == "bf16":
        pu.compare(type("W", (), {"dtype": DT[dtype]}), got, {n: want[n] for n in ("o", "lse", "dq", "dk", "dv")}, fp32=False)
        return
    for n in ("o", "dq", "dk", "dv"):
        assert np.all(np.isfinite(got[n]))
        assert np.all(np.abs(got[n] - want[n]) <= want["rel"] * want["size"][n] + 1e-30), n
    assert np.all(np.abs(got["lse"] - want["lse"]) <= want["rel"] * (1 + np.abs(want["lse"])))


def check(lens, H, dqk, dv, dtype, window, sinks, seed=0, scale=None, planned=True):
    q, k, v, do, offs = batch(lens, H, dqk, dv, dtype, seed)
    kw = dict(sinks=sinks, scale=scale)
    ws = jfa.workspace(jfa.params_for(q, k, v, offs, scale, True))
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, ws=ws, **kw)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    grads = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, ws=ws, **kw)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    if q.shape[0]:
        want = reference(*(f64(x) for x in (q, k, v, do)), lens, window, sinks,
                         float(np.float32(dqk ** -0.5 if scale is None else scale)))
        got = dict(zip(("o", "lse", "dq", "dk", "dv"), (f64(x) for x in (o, lse, *grads))))
        compare(got, want, dtype)
    if planned:  # one plan, several layers: the same bits
        jfa.jfa_window_plan(q, k, v, offs, window, ws=ws, **kw)
        for _ in range(2):
            o2, lse2 = jfa.jfa_window_fwd(q, k, v, offs, window, ws=ws, planned=True, **kw)
            g2 = jfa.jfa_window_bwd(q, k, v, o2, lse2, do, offs, window, ws=ws, planned=True, **kw)
            assert jfa.jfa_status_check(ws) == jfa.JFA_OK
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            for x, y in zip(grads, g2):
                assert torch.equal(x, y)
    return q, k, v, do, offs, o, lse, grads


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 300, 640]
CASES = [
    # lens, H, dqk, dv, dtype, window, sinks
    (EDGES, 2, 128, 128, "bf16", 1, 0),
    (EDGES, 2, 128, 128, "bf16", 1, 1),
    (EDGES, 2, 128, 128, "bf16", 100, 4),
    (EDGES, 1, 128, 128, "bf16", 128, 0),
    (EDGES, 1, 128, 128, "bf16", 129, 128),
    (EDGES, 1, 64, 64, "bf16", 2, 130),
    (EDGES, 3, 64, 64, "bf16", 65, 0),
    (EDGES, 2, 64, 64, "bf16", 200, 257),
    (EDGES, 2, 128, 64, "bf16", 127, 3),
    (EDGES, 2, 64, 128, "bf16", 300, 0),
    (EDGES, 2, 64, 128, "bf16", 17, 600),
    (EDGES, 2, 128, 128, "bf16", 5000, 0),
    ([1500, 3, 2000], 2, 128, 128, "bf16", 256, 4),
    ([4000], 1, 64, 64, "bf16", 1000, 1),
    ([1] * 300, 2, 128, 128, "bf16", 3, 1),
    (EDGES, 2, 32, 32, "f32", 1, 0),
    (EDGES, 2, 32, 32, "f32", 33, 2),
    (EDGES, 1, 100, 40, "f32", 64, 65),
    (EDGES, 2, 8, 8, "f32", 31, 0),
    (EDGES, 1, 128, 128, "f32", 400, 33),
    (EDGES, 2, 40, 24, "bf16", 50, 4),
]


@pytest.mark.parametrize("case", CASES, ids=["%dx%d-H%d-D%d-%d-%s-w%d-s%d" % (len(c[0]), max(c[0]), *c[1:]) for c in CASES])
def test_forward_and_backward(case):
    check(*case)


def test_many_items_a_cta():
    rng = np.random.default_rng(2)
    check(rng.integers(1, 300, 500).tolist(), 2, 128, 128, "bf16", 90, 4, planned=False)
    check(rng.integers(1, 300, 500).tolist(), 2, 64, 64, "bf16", 150, 0, planned=False)


@pytest.mark.parametrize("dim", [64, 128])
def test_a_window_of_everything_is_causal_attention(dim):
    q, k, v, do, offs = batch(EDGES, 2, dim, dim, "bf16")
    o, lse = jfa.jfa_fwd(q, k, v, offs, causal=True)
    g = jfa.jfa_bwd(q, k, v, o, lse, do, offs, causal=True)
    for window, sinks in ((640, 0), (2 ** 40, 0), (1, 640), (2 ** 31 - 1, 2 ** 31 - 1)):
        o2, lse2 = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks)
        g2 = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)
        for x, y in zip((o, lse, g[2]), (o2, lse2, g2[2])):
            assert torch.equal(x, y)
        # dS is rounded once here and three times there: each is within 1e-2 of the exact one
        for x, y in zip(g[:2], g2[:2]):
            assert float((x.float() - y.float()).norm() / x.float().norm()) <= 2e-2


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 40)])
def test_a_window_of_one_key_is_its_value(dtype, dim):
    q, k, v, do, offs = batch([5, 300, 64], 2, dim, dim, dtype)
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, 1)
    assert torch.equal(o, v)
    dq, dk, dv = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 1)
    if dtype == "bf16":
        # the weight exp2(s - lse) is 1 within fp32 roundings of both, which bf16 takes to 1
        assert torch.equal(dv, do)
    # dP - D is a sum of dim products minus the same sum: exact up to both sums' roundings
    size = (do.float().abs() * v.float().abs()).sum(-1, keepdim=True) * dim * 2.0 ** -22
    for g, x in ((dq, k), (dk, q)):
        bound = size * x.float().abs() * dim ** -0.5 * 1.1 + 1e-30
        assert bool((g.float().abs() <= bound).all())


def spiky(dtype, dim, size):
    lens = [700, 300]
    q, k, v, do, offs = batch(lens, 2, dim, dim, dtype, seed=4)
    at = torch.cat([torch.arange(n, device="cuda") for n in lens]) % 150
    k[(at >= 10) & (at < 30)] *= size
    return lens, q, k, v, do, offs, at


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("f32", 40)])
def test_hidden_scores_far_above_the_seen(dtype, dim):
    """Keys that score far above what rows behind their window see: nothing of them may remain."""
    window, sinks = 64, 3
    lens, q, k, v, do, offs, _ = spiky(dtype, dim, 20.0)
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks)
    grads = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)
    want = reference(*(f64(x) for x in (q, k, v, do)), lens, window, sinks, float(np.float32(dim ** -0.5)))
    compare(dict(zip(("o", "lse", "dq", "dk", "dv"), (f64(x) for x in (o, lse, *grads)))), want, dtype)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("f32", 40)])
def test_hidden_scores_of_any_size(dtype, dim):
    """Hidden scores of 10^30 leave the rows that do not see them as they are without those keys' size.  (The
    rows that see them have scores whose own fp32 rounding is 10^23: no backward is defined there.)"""
    window, sinks = 64, 3
    outs = []
    for size in (1.0, 1e30):
        _, q, k, v, _, offs, at = spiky(dtype, dim, size)
        outs.append(jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks))
    free = (at < 10) | (at >= 30 + window - 1)
    free[:30 + window] &= False  # (the first sequence's rows before any big key: nothing hidden)
    for a, b in zip(*outs):
        # the running maximum may move in other steps: fp32 sums, one rounding to bf16
        assert bool(torch.isfinite(b[free].float()).all())
        assert float((a[free].float() - b[free].float()).norm() / a[free].float().norm()) <= (2.0 ** -8 if a.dtype == torch.bfloat16 else 1e-5)


def test_gradient_against_differences():
    """Directional differences of the 64-bit forward (h = 1e-4: 1e-7 of the third derivative, 1e-12 / 1e-4 of
    cancellation) against the fp32 gradients, within their bound."""
    lens, H, D, window, sinks = [40, 7, 90], 2, 24, 13, 2
    q, k, v, do, offs = batch(lens, H, D, D, "f32", seed=3)
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks)
    grads = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)
    x = [f64(t) for t in (q, k, v)]
    d, scale = f64(do), float(np.float32(D ** -0.5))
    want = reference(*x, d, lens, window, sinks, scale)
    loss = lambda y: np.sum(d * reference(*y, d, lens, window, sinks, scale)["o"])
    rng = np.random.default_rng(0)
    for _ in range(6):
        u = [rng.standard_normal(t.shape) for t in x]
        h = 1e-4
        diff = (loss([a + h * b for a, b in zip(x, u)]) - loss([a - h * b for a, b in zip(x, u)])) / (2 * h)
        got = sum(np.sum(f64(g) * b) for g, b in zip(grads, u))
        noise = sum(np.sum(want["rel"] * want["size"][n] * np.abs(b)) for n, b in zip(("dq", "dk", "dv"), u))
        assert abs(got - diff) <= noise + 1e-4, (got, diff)


def test_streams_graphs_and_given_outputs():
    lens = [300, 0, 129, 50]
    q, k, v, do, offs = batch(lens, 2, 128, 128, "bf16")
    ws = jfa.workspace(jfa.params_for(q, k, v, offs, None, True))
    o, lse = torch.empty_like(v), torch.empty(q.shape[:2], device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def step():
        jfa.jfa_window_plan(q, k, v, offs, 70, sinks=4, ws=ws)
        jfa.jfa_window_fwd(q, k, v, offs, 70, sinks=4, o=o, lse=lse, ws=ws, planned=True)
        jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 70, sinks=4, dq=dq, dk=dk, dv=dv, ws=ws, planned=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([300, 0, 129, 50], [1, 400, 0, 78], [0, 0, 479, 0]):
        offs.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)])))
        for x in (q, k, v, do):
            x.normal_()
        g.replay()
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        want = reference(*(f64(x) for x in (q, k, v, do)), lens, 70, 4, float(np.float32(128 ** -0.5)))
        compare(dict(zip(("o", "lse", "dq", "dk", "dv"), (f64(x) for x in (o, lse, dq, dk, dv)))), want, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, _ = jfa.jfa_window_fwd(q, k, v, offs, 70, sinks=4, stream=s)
    s.synchronize()
    assert torch.equal(o, o2)


def test_invalid_offsets_compute_nothing():
    for dtype, dim in (("bf16", 64), ("f32", 32)):
        q, k, v, do, offs = batch([100, 50], 2, dim, dim, dtype)
        ws = jfa.workspace(jfa.params_for(q, k, v, offs, None, True))
        o, lse = torch.full_like(v, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        g = [torch.full_like(x, 7.0) for x in (q, k, v)]
        for bad in ([0, 151, 150], [1, 100, 150], [0, 100, 149]):
            b = torch.tensor(bad, device="cuda")
            jfa.jfa_window_fwd(q, k, v, b, 10, sinks=1, o=o, lse=lse, ws=ws)
            assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
            jfa.jfa_window_bwd(q, k, v, o, lse, do, b, 10, sinks=1, dq=g[0], dk=g[1], dv=g[2], ws=ws)
            assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
        for x in (o, lse, *g):
            assert bool((x == 7).all())


def test_a_wait_that_runs_out():
    q, k, v, do, offs = batch([300, 200], 2, 128, 128, "bf16")
    ws = jfa.workspace(jfa.params_for(q, k, v, offs, None, True))
    jfa.jfa_test_hold(True)
    try:
        jfa.jfa_window_fwd(q, k, v, offs, 50, sinks=2, ws=ws)
        st = jfa.jfa_status_check(ws)
    finally:
        jfa.jfa_test_hold(False)
    assert st == jfa.JFA_ERR_TIMEOUT
    check([300, 200], 2, 128, 128, "bf16", 50, 2)


def test_empty_batches():
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    for lens in ([], [0, 0]):
        offs = torch.zeros(len(lens) + 1, dtype=torch.int64, device="cuda")
        ws = jfa.workspace(jfa.params_for(e, e, e, offs, None, True))
        o, lse = jfa.jfa_window_fwd(e, e, e, offs, 5, ws=ws)
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK and o.shape == (0, 2, 64) and lse.shape == (0, 2)
        grads = jfa.jfa_window_bwd(e, e, e, o, lse, e, offs, 5, ws=ws)
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK and all(g.shape == e.shape for g in grads)
    offs = torch.tensor([0, 1], device="cuda")
    ws = jfa.workspace(jfa.params_for(e, e, e, offs, None, True))
    jfa.jfa_window_fwd(e, e, e, offs, 5, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS


def test_work_lists():
    """The lists' items and steps, from the definition of what a tile meets."""
    lens, H, window, sinks, tile = [700, 0, 1, 300, 129], 2, 150, 5, 128
    q, k, v, do, offs = batch(lens, H, 128, 128, "bf16")
    ws = jfa.jfa_window_plan(q, k, v, offs, window, sinks=sinks)
    torch.cuda.synchronize()
    hdr = ws[:256].cpu().numpy().view(np.int32)
    see = [wref.window_mask(np.arange(n), np.arange(n), window, sinks) for n in lens]
    cells = lambda b, rows, keys: see[b][rows * tile:(rows + 1) * tile, keys * tile:(keys + 1) * tile].any()
    tiles = [-(-n // tile) for n in lens]
    want_q = sorted((b, h, t, sum(cells(b, t, j) for j in range(tiles[b])))
                    for b in range(len(lens)) for h in range(H) for t in range(tiles[b]))
    want_k = []  # rows from the tile's own on, one stretch
    for b in range(len(lens)):
        for t in range(tiles[b]):
            met = [i for i in range(tiles[b]) if cells(b, i, t)]
            want_k += [(b, h, t, met[-1] - t + 1) for h in range(H)]
    off = 256
    up = lambda x: -(-x // 256) * 256
    off = up(up(off + 16 * len(lens)) + 16 * (len(lens) + 1))
    T = sum(lens)
    most = H * (T // 32 + len(lens) + 1)
    raw = ws.cpu().numpy()
    for n, want in ((hdr[1], want_q), (hdr[2], sorted(want_k))):
        items = raw[off:off + 32 * n].view(np.int32).reshape(-1, 8)
        assert sorted(tuple(int(y) for y in x[:4]) for x in items) == [tuple(int(y) for y in x) for x in want]
        off = up(off + 32 * most)


def test_refusals():
    q, k, v, do, offs = batch([10], 2, 64, 64, "bf16")
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, 4)
    for window, sinks in ((0, 0), (-3, 0), (4, -1)):
        for call in (lambda: jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks),
                     lambda: jfa.jfa_window_plan(q, k, v, offs, window, sinks=sinks),
                     lambda: jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)):
            with pytest.raises(ValueError):
                call()
    bad = [lambda: jfa.jfa_window_fwd(q, k[:5], v, offs, 4), lambda: jfa.jfa_window_fwd(q, k, v[:, :1], offs, 4),
           lambda: jfa.jfa_window_fwd(q, k, v.float(), offs, 4), lambda: jfa.jfa_window_fwd(q, k, v, offs.int(), 4),
           lambda: jfa.jfa_window_fwd(q[:, :, ::2], k[:, :, ::2], v, offs, 4), lambda: jfa.jfa_window_fwd(q, k, v, offs, 4, planned=True),
           lambda: jfa.jfa_window_fwd(q, k, v, offs, 4, o=q[:5]), lambda: jfa.jfa_window_bwd(q, k, v, o, lse, do[:4], offs, 4),
           lambda: jfa.jfa_window_bwd(q, k, v, o, lse.double(), do, offs, 4),
           lambda: jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 4, dk=q[:, :1])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(jfa.JfaError) as e:
        jfa.jfa_window_fwd(q, k, v, offs, 4, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == jfa.JFA_ERR_WORKSPACE
