"""Which sequences behind a shared prefix the kernel for few own keys takes, and results at its bounds.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_paged_gpu import f64
from test_shared_gpu import Shared, check, queries, space

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,own,few", [
    ("bf16", 2, True), ("bf16", 12, True), ("bf16", 13, False), ("bf16", 16, False), ("bf16", 17, False),
    ("mxfp8", 12, True), ("mxfp8", 13, True), ("mxfp8", 16, True), ("mxfp8", 17, False)])
def test_which_sequences_have_few_keys(kind, own, few):
    """Pages that may hold more than 16 keys: the tiled kernels' plan, in front of the workspace, is empty where the
    kernel for few keys takes every sequence."""
    n = 40
    b = Shared([n], [200], [1] * n, [own] * n, 2, 64, 64, 16, kind, "bf16", wide=True)
    assert b.own[1].shape[1] * 16 > 16
    ws = torch.zeros_like(space(b, 4))
    b.call(queries(b, 4), ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    assert (int(ws[256:260].cpu().numpy().view(np.int32)[0]) == n) == few


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("mxfp8", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("wide", [False, True])
def test_results_on_both_sides_of_the_bounds(kind, dtype, wide):
    n = 56
    own = np.array([11, 12, 13, 14, 15, 16, 17, 0])[np.arange(n) % 8]
    if not wide:
        own = np.minimum(own, 16)
    b = Shared([20, 36], [300, 77], (1 + np.arange(n) % 4).tolist(), own.tolist(), 2, 64, 64, 16, kind, dtype, wide=wide)
    for causal in (True, False):
        check(b, 8, causal)


@pytest.mark.parametrize("kind,dtype,dqk,dv", [("bf16", "bf16", 80, 80), ("bf16", "bf16", 64, 40), ("f32", "f32", 64, 64)])
@pytest.mark.parametrize("own,few", [(13, True), (16, True), (17, False)])
def test_which_sequences_have_few_keys_beside_cuda_cores(kind, dtype, dqk, dv, own, few):
    """CUDA cores take far longer a tile than the kernel for few keys: all up to 16 keys are its own there."""
    n = 40
    b = Shared([n], [70], [1] * n, [own] * n, 2, dqk, dv, 16, kind, dtype, wide=True)
    ws = torch.zeros_like(space(b, 4))
    check(b, 4, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    assert (int(ws[256:260].cpu().numpy().view(np.int32)[0]) == n) == few
