"""Planned calls on a plan that is another request's, or none: outputs are undefined, but nothing
outside them is touched and the next call is right (tests/test_paged_plan_cpu.py has the indexes on
the CPU).  GPU only."""
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_paged_gpu import DT, Batch, check_attention

pytestmark = pytest.mark.gpu

# new tokens, lengths, hq, hk, dtype: few rows, many rows, CUDA cores
REQUESTS = {
    "few": ([1] * 9, [300, 5, 64, 1, 700, 90, 33, 128, 20], 8, 4, "bf16"),
    "few of one head": ([1, 1, 2], [40, 700, 9], 8, 1, "bf16"),
    "many": ([300, 1, 77], [500, 20, 77], 8, 4, "bf16"),
    "many of one head": ([150, 40], [150, 1000], 4, 1, "bf16"),
    "CUDA cores": ([3, 1, 20], [300, 64, 20], 4, 2, "f32"),
}


def make(name):
    new, lens, hq, hk, dtype = REQUESTS[name]
    return Batch(new, lens, hk, 64, 64, 16, dtype, dtype, seed=len(name)), hq


@pytest.mark.parametrize("of", list(REQUESTS) + ["none"])
@pytest.mark.parametrize("name", list(REQUESTS))
def test_a_plan_that_does_not_fit_touches_nothing_else(name, of):
    b, hq = make(name)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    if of != "none":
        a, ha = make(of)
        jfa.jfa_paged_plan(torch.zeros(a.T, ha, 64, device="cuda", dtype=DT[a.dtype]), *a.args(), ws=ws)
    q = torch.randn(b.T, hq, 64, device="cuda").to(DT[b.dtype])
    guard = 1000
    o = torch.full((b.T + 2 * guard, hq, 64), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((b.T + 2 * guard, hq), 7.0, device="cuda")
    inner = slice(guard, guard + b.T)
    need = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, q.dtype, heads_q=hq)).numel()
    ws[need:] = 0x5a
    jfa.jfa_paged_fwd(q, *b.args(), ws=ws[:need], planned=True, o=o[inner], lse=lse[inner])
    torch.cuda.synchronize()
    for x in (o, lse):
        assert bool((x[:guard] == 7).all()) and bool((x[guard + b.T:] == 7).all())
    assert bool((ws[need:] == 0x5a).all())
    check_attention(b, hq, q=q, ws=ws[:need])
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
