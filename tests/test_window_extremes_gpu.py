"""Windows in training at the ends of the range: scores far below zero, and values and scores of hidden keys of any
size.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_window_gpu import DT, batch, f64, reference

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 128, 64), ("bf16", 64, 128), ("f32", 40, 40), ("bf16", 40, 24)]


def quiet(lens, H, dqk, dv, dtype, seed):
    """Scores that are integers around -1.56 million in log2 units (the scale makes one unit of q k one of those: ln 2
    in fp32 times log2 e is 1), but for loud keys, which score 0 to 3."""
    _, _, v, do, offs = batch(lens, H, dqk, dv, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = int(sum(lens))
    size = {128: 96, 64: 192, 40: 312}[dqk]  # bf16 holds them
    q = torch.full((T, H, dqk), 128.0, device="cuda")
    k = torch.full((T, H, dqk), -float(size), device="cuda")
    q[..., -1] = 1.0
    at = torch.cat([torch.arange(n, device="cuda") for n in lens])
    k[at % 97 == 50] = 0.0
    k[..., -1] = torch.randint(0, 4, (T, H), generator=g, device="cuda").float()
    return q.to(DT[dtype]), k.to(DT[dtype]), v, do, offs


@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 2), (64, 0), (130, 3), (400, 0), (1, 400)])
@pytest.mark.parametrize("dtype,dqk,dv", KINDS)
def test_seen_scores_far_below_zero(dtype, dqk, dv, window, sinks):
    """The hidden keys of a block, later sequences' among them, score as high as they like or as low."""
    lens, scale = [300, 5, 1, 200, 0, 130, 64], float(np.float32(np.log(2)))
    q, k, v, do, offs = quiet(lens, 2, dqk, dv, dtype, 7)
    kw = dict(sinks=sinks, scale=scale)
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, **kw)
    grads = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, **kw)
    want = reference(*(f64(x) for x in (q, k, v, do)), lens, window, sinks, scale)
    # Scores and their differences are exact, so weights are off by exp2 and their rounding to bf16, sums by fp32.
    one = 1.01 * 2.0 ** -8 if dtype == "bf16" else 0.0
    fp32 = 2.0 ** -23 * (max(lens) + 64)
    assert np.all(np.abs(f64(o) - want["o"]) <= (one + fp32) * want["size"]["o"] + one * np.abs(want["o"]))
    # lse: log2 units, its own rounding, ln 2 twice
    assert np.all(np.abs(f64(lse) - want["lse"]) <= 2.0 ** -22 * np.abs(want["lse"]) + 2.0 ** -20)
    # The backward takes the weights from lse: four roundings of 2^-24 of 1.57e6 log2 units, together at most 0.374,
    # a factor of 1.296 that all weights of a row share.
    for name, g in zip(("dq", "dk", "dv"), grads):
        assert bool(torch.isfinite(g.float()).all()), name
        tol = (0.296 + 4 * one + fp32) * want["size"][name]
        assert np.all(np.abs(f64(g) - want[name]) <= tol + 1e-30), name


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("f32", 100)])
def test_the_lowest_scores_under_one_window_of_everything(dtype, dim):
    """Every score is -16,384 dim: a window of one key returns its value, one of everything the mean so far (also
    behind the last sequence, where a tile's keys are the zeros past the buffer)."""
    lens = [300, 7, 129]
    q, k, v, _, offs = batch(lens, 2, dim, dim, dtype, seed=3)
    q.fill_(128.0)
    k.fill_(-128.0)
    low = -16384.0 * dim
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, 1, scale=1.0)
    assert torch.equal(o, v)
    assert bool(((lse - low).abs() <= 2.0 ** -21 * -low).all())
    # weights of a row are one number, rounded to bf16 for the product but not in their sum
    one = 1.01 * 2.0 ** -8 if dtype == "bf16" else 0.0
    for window, sinks in ((300, 0), (1, 300)):
        o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks, scale=1.0)
        for t, n in zip(np.cumsum([0] + lens), lens):
            x, count = f64(v[t:t + n]), np.arange(1, n + 1)[:, None, None]
            mean, size = np.cumsum(x, 0) / count, np.cumsum(np.abs(x), 0) / count
            assert np.all(np.abs(f64(o[t:t + n]) - mean) <= (one + 2.0 ** -23 * (n + 64)) * size + one * np.abs(mean))
            assert np.all(np.abs(f64(lse[t:t + n]) - low - np.log(count[..., 0])) <= 2.0 ** -21 * -low)


def loud_values(lens, window, sinks, dqk, dv, dtype, size):
    """Values of `size` at positions 10 to 29 of every sequence, gradients of 16 where rows do not see them, of 0
    where they do.  Returns which rows do not."""
    q, k, v, do, offs = batch(lens, 2, dqk, dv, dtype, seed=6)
    at = torch.cat([torch.arange(n, device="cuda") for n in lens])
    loud = (at >= 10) & (at < 30)
    free = (at < 10) | (at >= 29 + window)
    v[loud] = size
    do[free] = 16.0
    do[~free] = 0.0
    return q, k, v, do, offs, free


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 3), (140, 0), (5, 2), (128, 10)])
@pytest.mark.parametrize("dtype,dqk,dv", KINDS)
def test_gradients_beside_large_hidden_values(dtype, dqk, dv, window, sinks):
    """<dO, v> of hidden pairs is past fp32: nothing of it may reach the gradients."""
    lens = [300, 70, 450, 9]
    q, k, v, do, offs, free = loud_values(lens, window, sinks, dqk, dv, dtype, 2.0 ** 120)
    assert 16 * dv * 2 ** 120 > 2 ** 128
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks)
    grads = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)
    want = reference(*(f64(x) for x in (q, k, v, do)), lens, window, sinks, float(np.float32(dqk ** -0.5)))
    # weights, dS, o (in D) and the result, each rounded once; sums in fp32
    one = 1.01 * 2.0 ** -8 if dtype == "bf16" else 0.0
    for name, g in zip(("dq", "dk", "dv"), grads):
        g = f64(g)
        assert np.all(np.isfinite(g)), name
        assert np.all(np.abs(g - want[name]) <= (3 * one + want["rel"]) * want["size"][name] + one * np.abs(want[name]) + 1e-30), name


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 3), (1, 0), (5, 2), (128, 10)])
@pytest.mark.parametrize("dtype,dqk,dv", KINDS)
def test_outputs_beside_the_largest_hidden_values(dtype, dqk, dv, window, sinks):
    lens = [300, 70, 450, 9]
    outs = []
    for size in (0.0, 3e38):
        q, k, v, _, offs, free = loud_values(lens, window, sinks, dqk, dv, dtype, size)
        outs.append(jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks))
    for a, b in zip(*outs):
        assert torch.equal(a[free], b[free])
