"""The rotation's angles against frequencies in 60 digits: within fp32 rounding for the positions of
any context, and within |pos| 2^-53 turns for far ones, as stated in include/jfa.h.  GPU only."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref
from test_norm_rope_gpu import FWD

pytestmark = pytest.mark.gpu

TURN = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
# Of a frequency, relative: pow (2^-52) of an exponent rounded by 2^-53 (times the power's
# logarithm, at most ln(500000)), a division by the rounded 2 pi (2^-53 and 2^-54), another by the factor.
# Turns are at most 1 / 2 pi, and e^-u (u + 5) at most 5: 5 / 6.28 * 2^-53.
PER_POSITION = 2.0 ** -53


def turns(rot, base, scaling, factor, orig_len=4096, fast=32, slow=1):
    """Turns a position of every pair."""
    getcontext().prec = 60
    b, f = Decimal(base), Decimal(factor)
    if scaling == "ntk":
        b *= ((Decimal(rot) / (rot - 2)) * f.ln()).exp()
    out = []
    for i in range(rot // 2):
        t = ((Decimal(-2 * i) / rot) * b.ln()).exp() / TURN
        if scaling == "linear":
            t /= f
        if scaling == "yarn":
            g = min(Decimal(1), max(Decimal(0), (orig_len * t - slow) / (fast - slow)))
            t *= g + (1 - g) / f
        out.append(t)
    return out


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 40])
@pytest.mark.parametrize("rot,base,scaling,factor", [(64, 10000, "none", 1), (128, 500000, "none", 1), (48, 10000, "linear", 3),
                                                     (64, 10000, "ntk", 8), (128, 10000, "yarn", 16)])
def test_angles(rot, base, scaling, factor, far):
    T = 60
    rng = np.random.default_rng(rot)
    pos = np.concatenate([rng.integers(0, far, T - 4), [0, 1, -1, -far]])
    x = rng.standard_normal((T, 2, rot)).astype(np.float32)
    rope = jfa.jfa_rope(rot, base=float(base), scaling=scaling, factor=float(factor), orig_len=4096.0)
    y, _ = jfa.jfa_norm_rope_fwd(torch.tensor(x, device="cuda"), None, torch.tensor(pos, device="cuda"), rope=rope, norm=False)
    at = [[float(int(p) * t % 1 * TURN) for t in turns(rot, base, scaling, factor)] for p in pos]
    c, s = np.cos(at)[:, None], np.sin(at)[:, None]
    x = x.astype(np.float64)
    a, b = x[..., :rot // 2], x[..., rot // 2:]
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    tol = (FWD + 6.3 * PER_POSITION * np.abs(pos.astype(np.float64))[:, None, None]) * ref._reach(x, rot, "halves", 1.0)
    tol = tol + ref.HALF_STEP["f32"] * np.abs(want)
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / tol))
