"""Cosines and sines of the rotation, of queries and of keys on their way to a cache, within fp32's own steps at every
angle: also near half turns and quarter turns, where one of them is small.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_norm_rope_angles_gpu import PER_POSITION, TURN, turns

pytestmark = pytest.mark.gpu


def compare(got, pos, rot, base):
    """got [T, rot]: (1, 0) turned.  What the angle is off: 2^-24 of its distance to the nearest quarter turn (one
    rounding), the phase's step of 2^-32 turns, and the frequency's error.  sincospif is within 2 ulp."""
    f = turns(rot, base, "none", 1)
    exact = np.array([[float(int(p) * t % 1) for t in f] for p in pos])
    left = np.abs(exact - np.round(exact * 4) / 4) * float(TURN)
    c, s = np.cos(exact * float(TURN)), np.sin(exact * float(TURN))
    # (where an angle is next to a quarter turn 64 bits' own cosine or sine is off by 2^-53 of a turn's angle)
    angle = 2.0 ** -24 * left + float(TURN) * (2.0 ** -32 + PER_POSITION * np.abs(pos)[:, None].astype(float)) + 2.0 ** -50
    got = got.astype(np.float64)
    for x, want, slope in ((got[:, :rot // 2], c, np.abs(s)), (got[:, rot // 2:], s, np.abs(c))):
        tol = angle * slope + angle ** 2 + 2.0 ** -22 * np.abs(want)
        worst = np.abs(x - want) / tol
        assert np.max(worst) <= 1, (float(np.max(worst)), np.unravel_index(np.argmax(worst), worst.shape))
    return left


@pytest.mark.parametrize("rot,base", [(64, 10000), (128, 500000)])
def test_cosines_and_sines(rot, base):
    T = 3000
    rng = np.random.default_rng(rot)
    pos = np.concatenate([rng.integers(0, 10 ** 5, T - 3), [0, 1, -1]])
    x = torch.zeros(T, 1, rot, device="cuda")
    x[..., :rot // 2] = 1.0
    p, rope = torch.tensor(pos, device="cuda"), jfa.jfa_rope(rot, base=float(base))
    y, _ = jfa.jfa_norm_rope_fwd(x, None, p, rope=rope, norm=False)
    left = compare(y[:, 0].cpu().numpy(), pos, rot, base)
    assert (left < 1e-3).sum() > 100  # angles next to quarter turns are among them
    # keys, and queries beside them, appended to a cache
    cache = jfa.paged_cache(-(-T // 64), 1, rot, page_size=64, dtype=torch.float32)
    table = torch.arange(-(-T // 64), device="cuda").int()[None].contiguous()
    offs, lens = torch.tensor([0, T], device="cuda"), torch.tensor([T], device="cuda")
    yq, ws = jfa.jfa_rope_append(x, x, x, cache, table, offs, lens, rope=rope, norm=False, pos=p)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    k, _ = jfa.jfa_cache_read(cache, table, offs, lens, T, dtype=torch.float32)
    assert torch.equal(yq, y) and torch.equal(k, y)
