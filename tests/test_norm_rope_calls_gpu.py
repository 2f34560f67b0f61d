"""Calls of the norm with rotary positions that leave arguments out.  GPU only."""
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_norm_rope_gpu import inputs

pytestmark = pytest.mark.gpu


def test_no_positions_where_nothing_turns():
    q, k, pos, wq, wk, dyq, dyk = inputs(7, 2, 1, 64, "bf16")
    still = jfa.jfa_rope(0)
    for rope in (None, still):
        got = jfa.jfa_norm_rope_fwd(q, k, None, wq, wk, rope=rope)
        want = jfa.jfa_norm_rope_fwd(q, k, pos, wq, wk, rope=still)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = jfa.jfa_norm_rope_bwd(q, k, None, dyq, dyk, wq, wk, rope=rope)
        want = jfa.jfa_norm_rope_bwd(q, k, pos, dyq, dyk, wq, wk, rope=still)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_missing_tensors_are_refused():
    q, k, pos, wq, wk, dyq, dyk = inputs(7, 2, 1, 64, "bf16")
    for bad in (lambda: jfa.jfa_norm_rope_fwd(q, k, None, wq, wk, rope=jfa.jfa_rope(64)),
                lambda: jfa.jfa_norm_rope_bwd(q, k, pos, None, dyk, wq, wk, rope=jfa.jfa_rope(64)),
                lambda: jfa.jfa_norm_rope_bwd(q, k, pos, dyq, None, wq, wk, rope=jfa.jfa_rope(64))):
        with pytest.raises(ValueError):
            bad()
