"""Norms of query and key heads with rotary positions (jfa_norm_rope_fwd / _bwd) against the
definition in 64 bits, element by element.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# Error of a value before its last rounding, relative to the size of what it is computed from:
# a row's sum of squares, D <= 256 fp32 terms in chains of at most 24, is within 1.5e-6, r half of
# that plus 2.4e-7 (rsqrtf), three products 1.8e-7, cos and sin 2.2e-7 each (the angle's
# rounding to 2^-25 half turns times pi, two units of sincospif), their two products 1.2e-7.
FWD = 2e-6
# The backward also has the row's <u, x> (as the sum of squares), r three times and two products
# more.
BWD = 5e-6


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(T, hq, hk, D, dtype, seed=0, far=5000, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    if fused:  # slices of a projection's output, with the values behind them
        x = (rn(T, hq + 2 * hk, D) * torch.exp(rn(T, hq + 2 * hk, 1))).to(DT[dtype])
        q, k = x[:, :hq], x[:, hq:hq + hk]
    else:
        q = (rn(T, hq, D) * torch.exp(rn(T, hq, 1))).to(DT[dtype]) if hq else None
        k = (rn(T, hk, D) * torch.exp(rn(T, hk, 1))).to(DT[dtype]) if hk else None
    pos = torch.randint(0, far, (T,), generator=g, device="cuda")
    dyq = rn(T, hq, D).to(DT[dtype]) if hq else None
    dyk = rn(T, hk, D).to(DT[dtype]) if hk else None
    return q, k, pos, 1 + 0.3 * rn(D), 1 + 0.3 * rn(D), dyq, dyk


CASES = [
    # T, hq, hk, D, rot, layout, dtype, rope keywords, fused
    (1, 1, 1, 128, 128, "halves", "bf16", {}, False),
    (67, 8, 2, 128, 128, "halves", "bf16", {}, True),
    (67, 8, 2, 128, 128, "pairs", "bf16", {}, True),
    (33, 3, 1, 64, 32, "halves", "bf16", dict(scaling="linear", factor=4.0), False),
    (33, 5, 5, 96, 48, "pairs", "f32", dict(scaling="ntk", factor=8.0), True),
    (41, 7, 1, 80, 16, "halves", "f32", dict(scaling="yarn", factor=16.0, orig_len=2048.0, amp=1.3), False),
    (19, 2, 3, 256, 256, "pairs", "bf16", dict(base=500000.0), False),
    (300, 32, 8, 128, 64, "halves", "f32", {}, True),
    (9, 2, 2, 16, 16, "pairs", "bf16", {}, False),
    # rows without whole slots: single values
    (13, 3, 2, 20, 12, "halves", "bf16", {}, False),
    (13, 3, 2, 33, 20, "pairs", "f32", {}, True),
    (5, 1, 4, 250, 250, "halves", "f32", {}, False),
    (7, 2, 1, 128, 4, "halves", "bf16", dict(scaling="ntk", factor=2.0), False),
    (3, 1, 1, 1, 0, "halves", "f32", None, False),
    # one tensor, no rotation
    (21, 4, 0, 64, 64, "halves", "bf16", {}, False),
    (21, 0, 4, 64, 0, "halves", "f32", None, False),
]


def rope_of(rot, layout, kw):
    if kw is None:
        return None, np.zeros(0), 1.0
    freq = ref.frequencies(rot, **{a: b for a, b in kw.items() if a != "amp"})
    return jfa.jfa_rope(rot, layout=layout, **kw), freq, kw.get("amp", 1.0)


def check(got, want, size, unit, dtype, what):
    err = np.abs(f64(got) - want)
    tol = ref.HALF_STEP[dtype] * np.abs(want) * 1.01 + unit * size + 1e-36
    assert np.all(err <= tol), (what, float(np.max(err / tol)))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=["%d-%d-%d-D%d-r%d-%s-%s" % c[:7] for c in CASES])
def test_forward_and_backward(case, norm):
    T, hq, hk, D, rot, layout, dtype, kw, fused = case
    q, k, pos, wq, wk, dyq, dyk = inputs(T, hq, hk, D, dtype, fused=fused)
    rope, freq, amp = rope_of(rot, layout, kw)
    if rope is None:
        rot = 0
    w = dict(wq=wq if hq else None, wk=wk if hk else None) if norm else {}
    yq, yk = jfa.jfa_norm_rope_fwd(q, k, pos, rope=rope, eps=1e-5, norm=norm, **w)
    dq, dk, dwq, dwk = jfa.jfa_norm_rope_bwd(q, k, pos, dyq, dyk, rope=rope, eps=1e-5, norm=norm, **w)
    for x, wt, y, dy, dx, dw in ((q, wq, yq, dyq, dq, dwq), (k, wk, yk, dyk, dk, dwk)):
        if x is None:
            assert y is None and dx is None
            continue
        a = (f64(x), f64(wt) if norm else None, f64(pos), freq, rot, layout, amp, 1e-5)
        want, size = ref.norm_rope(*a, norm=norm)
        check(y, want, size, FWD, dtype, "y")
        want, wdw, size, sdw = ref.norm_rope_bwd(*a, f64(dy), norm=norm)
        check(dx, want, size, BWD, dtype, "dx")
        if norm:
            # a chain of at most 100 fp32 additions: rows of a lane, lanes, warps, CTAs
            err = np.abs(f64(dw) - wdw)
            assert np.all(err <= (BWD + 100 * ref.F32) * sdw), float(np.max(err / sdw))


def test_long_sum_of_weight_gradients_repeats():
    """Many tokens: the same bits twice, and the sum in its bound (chains of at most 2000)."""
    T, hq, hk, D = 30011, 4, 2, 64
    q, k, pos, wq, wk, dyq, dyk = inputs(T, hq, hk, D, "bf16", seed=3)
    rope, freq, amp = rope_of(D, "halves", {})
    runs = [jfa.jfa_norm_rope_bwd(q, k, pos, dyq, dyk, wq, wk, rope=rope) for _ in range(2)]
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    _, want, _, size = ref.norm_rope_bwd(f64(q), f64(wq), f64(pos), freq, D, "halves", amp, 1e-6, f64(dyq))
    assert np.all(np.abs(f64(runs[0][2]) - want) <= (BWD + 2000 * ref.F32) * size)


def test_gradient_against_differences():
    """Directional differences of the 64-bit forward: h = 1e-5, so 1e-9 of the third derivative
    and 1e-11 of cancellation; the kernel's fp32 gradient is within 1e-5 of its sizes."""
    T, H, D, rot = 6, 2, 48, 32
    q, k, pos, wq, wk, dyq, dyk = inputs(T, H, H, D, "f32", seed=5, far=200)
    rope, freq, amp = rope_of(rot, "pairs", dict(amp=0.7))
    dq, _, dwq, _ = jfa.jfa_norm_rope_bwd(q, k, pos, dyq, dyk, wq, wk, rope=rope, eps=1e-3)
    x, w, dy = f64(q), f64(wq), f64(dyq)
    loss = lambda x, w: np.sum(dy * ref.norm_rope(x, w, f64(pos), freq, rot, "pairs", amp, 1e-3)[0])
    rng = np.random.default_rng(0)
    for _ in range(8):
        a, b = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        h = 1e-5
        want = (loss(x + h * a, w + h * b) - loss(x - h * a, w - h * b)) / (2 * h)
        got = np.sum(f64(dq) * a) + np.sum(f64(dwq) * b)
        size = np.sum(np.abs(f64(dq) * a)) + np.sum(np.abs(f64(dwq) * b))
        assert abs(got - want) <= 1e-5 * size + 1e-7


def test_far_and_negative_positions():
    """Positions up to 2^40 and below zero.  The reference angle is exact: position times the
    64-bit fraction of a turn in integers."""
    T, D = 64, 64
    q, _, _, wq, _, _, _ = inputs(T, 2, 0, D, "f32", seed=1)
    rng = np.random.default_rng(1)
    pos = np.concatenate([rng.integers(-10 ** 6, 0, 16), rng.integers(0, 10 ** 9, 16),
                          rng.integers(2 ** 39, 2 ** 40, 30), [0, -1]])
    y, _ = jfa.jfa_norm_rope_fwd(q, None, torch.tensor(pos, device="cuda"), wq, rope=jfa.jfa_rope(D))
    n = f64(q) / np.sqrt(np.mean(f64(q) ** 2, -1, keepdims=True) + 1e-6) * f64(wq)
    turns = [10000.0 ** (-2.0 * i / D) / 6.283185307179586476925286766559 for i in range(D // 2)]
    frac = np.array([[(int(p) * int(t * 2.0 ** 64)) % 2 ** 64 / 2.0 ** 64 for t in turns] for p in pos])
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    a, b = n[..., :D // 2], n[..., D // 2:]
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    check(y, want, ref._reach(n, D, "halves", 1.0), FWD, "f32", "y")


def test_in_place_strides_and_untouched_neighbours():
    """Into the projection's own buffer, the values behind the heads as they were, and the
    backward into the gradient's buffer."""
    T, hq, hk, D = 37, 4, 2, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, hq + 2 * hk, D, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, hq + 2 * hk, D, generator=g, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda")
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    rope = jfa.jfa_rope(D)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    want = jfa.jfa_norm_rope_fwd(q, k, pos, w, w, rope=rope)
    wd = jfa.jfa_norm_rope_bwd(q, k, pos, dy[:, :hq], dy[:, hq:hq + hk], w, w, rope=rope)
    d2 = dy.clone()
    got = jfa.jfa_norm_rope_bwd(q, k, pos, d2[:, :hq], d2[:, hq:hq + hk], w, w, rope=rope, dq=d2[:, :hq],
                                dk=d2[:, hq:hq + hk])
    for a, b in zip(got, wd):
        assert torch.equal(a, b)
    assert torch.equal(d2[:, hq + hk:], dy[:, hq + hk:])
    y = x.clone()
    jfa.jfa_norm_rope_fwd(y[:, :hq], y[:, hq:hq + hk], pos, w, w, rope=rope, yq=y[:, :hq], yk=y[:, hq:hq + hk])
    assert torch.equal(y[:, :hq], want[0]) and torch.equal(y[:, hq:hq + hk], want[1])
    assert torch.equal(y[:, hq + hk:], x[:, hq + hk:])


def test_no_tokens_and_graph_replay():
    D = 64
    e = torch.empty(0, 2, D, device="cuda")
    w = torch.ones(D, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    yq, yk = jfa.jfa_norm_rope_fwd(e, e, pos, w, w, rope=jfa.jfa_rope(D))
    assert yq.shape == e.shape
    _, _, dwq, dwk = jfa.jfa_norm_rope_bwd(e, e, pos, e, e, w, w, rope=jfa.jfa_rope(D),
                                           dwq=torch.full_like(w, 7), dwk=torch.full_like(w, 7))
    assert torch.equal(dwq, torch.zeros_like(w)) and torch.equal(dwk, torch.zeros_like(w))

    q, k, pos, wq, wk, dyq, dyk = inputs(50, 4, 2, D, "bf16")
    rope = jfa.jfa_rope(D)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    bufs = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k),
            torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]

    def step():
        jfa.jfa_norm_rope_fwd(q, k, pos, wq, wk, rope=rope, yq=bufs[0], yk=bufs[1])
        jfa.jfa_norm_rope_bwd(q, k, pos, dyq, dyk, wq, wk, rope=rope, dq=bufs[2], dk=bufs[3], dwq=bufs[4],
                              dwk=bufs[5], ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q2, k2, pos2, _, _, dyq2, dyk2 = inputs(50, 4, 2, D, "bf16", seed=9)
    for a, b in ((q, q2), (k, k2), (pos, pos2), (dyq, dyq2), (dyk, dyk2)):
        a.copy_(b)
    graph.replay()
    want = [*jfa.jfa_norm_rope_fwd(q2, k2, pos2, wq, wk, rope=rope),
            *jfa.jfa_norm_rope_bwd(q2, k2, pos2, dyq2, dyk2, wq, wk, rope=rope)]
    for a, b in zip(bufs, want):
        assert torch.equal(a, b)


def test_nan_and_infinity_stay_in_their_row():
    q, _, pos, wq, _, _, _ = inputs(20, 3, 0, 64, "bf16")
    clean, _ = jfa.jfa_norm_rope_fwd(q, None, pos, wq, rope=jfa.jfa_rope(64))
    q[4, 1, 7], q[9, 2, 0] = float("nan"), float("inf")
    y, _ = jfa.jfa_norm_rope_fwd(q, None, pos, wq, rope=jfa.jfa_rope(64))
    keep = torch.ones(20, 3, dtype=torch.bool, device="cuda")
    keep[4, 1] = keep[9, 2] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[4, 1]).all()) and bool(torch.isnan(y[9, 2]).any())


def test_refused_tensors():
    q, k, pos, wq, wk, dyq, dyk = inputs(10, 2, 2, 64, "bf16")
    r = jfa.jfa_rope(64)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(None, None, pos, rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q.cpu(), None, pos.cpu(), rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q, k.float(), pos, rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q, k[:9], pos, rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q, k, pos.int(), rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q.transpose(1, 2), None, pos, rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q, k, pos, wq.bfloat16(), wk, rope=r)
    with pytest.raises(ValueError):
        jfa.jfa_norm_rope_fwd(q, k, pos, wq, wk, rope=r, norm=False)
    with pytest.raises(jfa.JfaError):  # a broadcast tensor's tokens share their memory
        jfa.jfa_norm_rope_fwd(q, q[:1].expand(10, 2, 64), pos, wq, wk, rope=r)
    with pytest.raises(jfa.JfaError):
        jfa.jfa_norm_rope_fwd(q, k, pos, rope=jfa.jfa_rope(66))
    with pytest.raises(TypeError):
        jfa.jfa_norm_rope_fwd(q.half(), k.half(), pos, rope=r)
