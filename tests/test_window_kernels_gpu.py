"""Which kernel serves a window over a paged cache: the plan's cuts, one for each CTA, tell.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa

pytestmark = pytest.mark.gpu


def shares(window, sinks, tokens, mxfp8=False):
    """How many CTAs a plan of 16 users' `tokens` tokens, 8 heads a key head, over 9,000 keys cuts its work for."""
    B, n, hk, page = 16, 9000, 8, 64
    per = -(-n // page)
    cache = jfa.paged_cache(B * per, hk, 128, page_size=page, mxfp8=mxfp8)
    table = torch.arange(B * per, device="cuda").int().view(B, per)
    q = torch.zeros(B * tokens, 8 * hk, 128, device="cuda", dtype=torch.bfloat16)
    offs, lens = torch.arange(B + 1, device="cuda") * tokens, torch.full((B,), n, device="cuda")
    ws = torch.zeros_like(jfa.jfa_paged_window_plan(q, cache, table, offs, lens, window, sinks=sinks))
    jfa.jfa_paged_window_plan(q, cache, table, offs, lens, window, sinks=sinks, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    pos = ws[256:256 + 16 * 1024].cpu().numpy().view(np.int32).reshape(-1, 4)
    return int(np.argmax(pos[:, 0] == B))  # the first place behind the batch


@pytest.mark.parametrize("window,sinks,tokens,few", [
    (64, 4, 3, True), (512, 0, 4, True), (64, 448, 3, True), (512, 0, 6, False), (600, 0, 3, False),
    (64, 8192, 3, False), (64, 8192, 4, False), (1, 2 ** 31 - 1, 3, False), (2 ** 31 - 1, 0, 3, False), (64, 8192, 2, True)])
def test_sinks_count_like_the_window(window, sinks, tokens, few):
    """16 to 48 rows a key head: the kernel of few rows, with two CTAs an SM, up to 16 rows, and up to 32 over at most
    512 keys of window and sinks; else the one of 128-row tiles, with one."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = shares(window, sinks, tokens)
    assert (n > sms) == few, n
