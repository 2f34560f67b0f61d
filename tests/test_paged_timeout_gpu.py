"""The bounded waits of the paged attention's tensor-core kernels give up cleanly.

jfa_test_hold makes one role of the first CTA wait on a barrier that nothing arrives on, with the
CTA's loads (and the other stream's MMAs) in flight.  After about two seconds it records
JFA_ERR_TIMEOUT and raises the CTA's abort flag; every other role has to leave its wait, the copies
have to land, and the next call on the same workspace has to be right.  GPU only."""
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_paged_gpu import Batch, _poisoned, check_attention

pytestmark = pytest.mark.gpu

KERNELS = [("few", "bf16", 8), ("few", "mxfp8", 8), ("few", "mxfp8", 32), ("many", "bf16", 8), ("many", "mxfp8", 8)]


def held(kind, cache, hq):
    """A batch in which every CTA has work, and its workspace."""
    if kind == "few":
        b = Batch([1, 2, 1], [9000, 5000, 7000], 2, 128, 128, 64, cache, "bf16")
    else:
        b = Batch([700, 300], [900, 3000], 2, 128, 128, 64, cache, "bf16")
    return b, jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, torch.bfloat16, heads_q=hq))


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("kind,cache,hq", KERNELS)
def test_a_wait_that_runs_out(kind, cache, hq, planned):
    b, ws = held(kind, cache, hq)
    q = torch.randn(b.T, hq, 128, device="cuda").bfloat16()
    o, lse = _poisoned(b, hq)
    if planned:
        jfa.jfa_paged_plan(q, *b.args(), ws=ws)
    jfa.jfa_test_hold(True)
    try:
        jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws, planned=planned)
        st = jfa.jfa_status_check(ws)
    finally:
        jfa.jfa_test_hold(False)
    assert st == jfa.JFA_ERR_TIMEOUT, jfa.status_string(st)
    if planned:
        jfa.jfa_paged_plan(q, *b.args(), ws=ws)
    check_attention(b, hq, q=q, ws=ws, planned=planned)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("kind,cache,hq", KERNELS)
def test_a_timeout_is_reported_ahead_of_bad_pages(kind, cache, hq, planned):
    """A bad page says that everything else was computed, so an incomplete call must not report one:
    bad pages in the first CTA's sequence and in others'."""
    b, ws = held(kind, cache, hq)
    b.table[0, 3] = -1
    b.table[1, 5] = b.pages
    q = torch.randn(b.T, hq, 128, device="cuda").bfloat16()
    if planned:
        jfa.jfa_paged_plan(q, *b.args(), ws=ws)
    jfa.jfa_paged_fwd(q, *b.args(), ws=ws, planned=planned)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
    jfa.jfa_test_hold(True)
    try:
        jfa.jfa_paged_fwd(q, *b.args(), ws=ws, planned=planned)
        st = jfa.jfa_status_check(ws)
    finally:
        jfa.jfa_test_hold(False)
    assert st == jfa.JFA_ERR_TIMEOUT, jfa.status_string(st)
