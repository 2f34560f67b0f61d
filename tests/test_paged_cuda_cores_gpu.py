"""bf16 attention at head dims that the CUDA-core kernel serves: its weights stay fp32, so its results
have no room for weights in bf16.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref
from test_paged_gpu import Batch, f64, ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["step", "chunk", "prompt", "one long", "many short"])
@pytest.mark.parametrize("cache,hq,hk,dqk,dv", [("bf16", 4, 2, 72, 8), ("bf16", 6, 2, 80, 80), ("mxfp8", 4, 1, 96, 96),
                                                ("mxfp8", 2, 2, 32, 128), ("bf16", 40, 2, 128, 96)])
def test_weights_are_not_rounded(kind, cache, hq, hk, dqk, dv):
    b = Batch(*ragged(kind), hk, dqk, dv, 32, cache, "bf16", seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(b.T, hq, dqk, generator=g, device="cuda").bfloat16()
    o, lse = jfa.jfa_paged_fwd(q, *b.args())
    wo, wl, av, size = ref.paged(f64(q), b.k_of, b.v_of, b.offs_h, b.lens_h, hq // hk, float(np.float32(dqk ** -0.5)), True)
    _, tl = ref.paged_bounds(wo, wl, av, size, dqk, 512, "bf16", False)
    # a score's error and exp2's (as there); a chain of one fused product and sum a key, its
    # rescaling by the maximum every 32 keys, the parts' join: 1.2 units of 2^-24 a key on either side
    # of the division; the result's own rounding
    ds = tl  # which has 1024 units for the sums of the lse
    keys = 2.4 * int(b.lens_h.max()) * ref.F32
    tol = (2 * ds + keys)[..., None] * av + ref.HALF_STEP["bf16"] * np.abs(wo) * 1.01 + 1e-30
    err = np.abs(f64(o) - wo)
    assert np.all(err <= tol), float(np.max(err / tol))
    fin = np.isfinite(wl)
    assert np.array_equal(fin, np.isfinite(f64(lse)))
    assert np.all(np.abs(f64(lse)[fin] - wl[fin]) <= tl[fin] + keys)
