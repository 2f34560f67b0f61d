"""Calls on the paged cache that have no new tokens: invalid batches are reported all the same.  GPU only."""
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_paged_gpu import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["none", "offsets", "negative", "long", "empty batch"])
@pytest.mark.parametrize("call", ["write", "read", "attention"])
def test_invalid_batches_without_tokens(what, call):
    b = Batch([] if what == "empty batch" else [0, 0, 0], [] if what == "empty batch" else [5, 0, 40], 2, 64, 64, 16, "bf16", "bf16")
    if what in ("offsets", "empty batch"):
        b.offs[-1] = 3
    elif what == "negative":
        b.lens[1] = -1
    elif what == "long":
        b.lens[2] = b.table.shape[1] * 16 + 1
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, 0, torch.bfloat16))
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = b.cache.k.view(torch.int16).clone()
    if call == "write":
        jfa.jfa_cache_write(none, none, *b.args(), ws=ws)
    elif call == "read":
        jfa.jfa_cache_read(*b.args(), 0, ws=ws)
    else:
        jfa.jfa_paged_fwd(none, *b.args(), ws=ws)
    assert jfa.jfa_status_check(ws) == (jfa.JFA_OK if what == "none" else jfa.JFA_ERR_BAD_OFFSETS)
    assert torch.equal(before, b.cache.k.view(torch.int16))
