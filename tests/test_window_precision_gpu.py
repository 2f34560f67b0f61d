"""How far the bf16 gradients under a window are off where rows see few keys.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_window_gpu import batch, f64, reference

pytestmark = pytest.mark.gpu

# One rounding to bf16 is uniform within half a step of 2^-7 of the value's power of two: 2^-8 / sqrt(3) of that
# in the mean square, and over mantissas as frequent as 1 / m in [1, 2) sqrt(3 / (8 ln 2)) of it relative to the
# value, 1.66e-3.  dS and the results are rounded, independently: 2.35e-3.  A quarter more for the sums' other errors
# and the scatter of norms over tens of thousands of elements.
BOUND = 1.25 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * (3 / (8 * np.log(2))) ** 0.5

LENS = [300, 0, 1, 2, 15, 16, 17, 31, 33, 257, 48]


@pytest.mark.parametrize("dqk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("window,sinks", [(2, 0), (3, 0), (5, 3), (1, 2), (10, 6), (1, 15), (16, 0), (9, 0), (17, 0), (2, 130)])
def test_gradients_of_rows_that_see_few_keys(window, sinks, dqk, dv):
    q, k, v, do, offs = batch(LENS, 3, dqk, dv, "bf16")
    o, lse = jfa.jfa_window_fwd(q, k, v, offs, window, sinks=sinks)
    dq, dk, _ = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, window, sinks=sinks)
    want = reference(*(f64(x) for x in (q, k, v, do)), LENS, window, sinks, float(np.float32(dqk ** -0.5)))
    for name, got in (("dq", dq), ("dk", dk)):
        err = np.linalg.norm(f64(got) - want[name]) / np.linalg.norm(want[name])
        assert err <= BOUND, (name, err)


def test_many_sequences():
    """More sequences than the row pass has CTAs, and one sequence alone that fills them."""
    for lens in ([3, 1, 40] * 1500, [20000]):
        q, k, v, do, offs = batch(lens, 1, 64, 64, "bf16")
        o, lse = jfa.jfa_window_fwd(q, k, v, offs, 4, sinks=1)
        dq, dk, _ = jfa.jfa_window_bwd(q, k, v, o, lse, do, offs, 4, sinks=1)
        some = lens if len(lens) > 1 else [2000]  # of the long one, rows whose window lies in front of the cut
        n = sum(some)
        want = reference(*(f64(x[:n]) for x in (q, k, v, do)), some, 4, 1, 0.125)
        n -= 4 if len(lens) == 1 else 0
        err = np.linalg.norm(f64(dq[:n]) - want["dq"][:n]) / np.linalg.norm(want["dq"][:n])
        assert err <= BOUND, err
