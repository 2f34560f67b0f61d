"""Plain 64-bit attention under any visibility, for windows and shared prefixes, and batches over a
paged cache whose hidden positions are poisoned.  numpy only, but for the batches."""
from __future__ import annotations

import math

import numpy as np

import serve_ref as ref


def window_mask(rows, keys, window, sinks):
    """Which key positions the query positions see."""
    i, j = np.asarray(rows)[:, None], np.asarray(keys)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def attend(q, seqs, group, scale, dv):
    """q [T, Hq, D]; seqs: of every sequence (first token, k [Hk, n, D], v [Hk, n, Dv], see [L, n]).
    Returns o, lse, sum p |v| and the largest scale sum |q k| of every row, as serve_ref.paged."""
    T, Hq, _ = q.shape
    o, av = np.zeros((T, Hq, dv)), np.zeros((T, Hq, dv))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for t0, k, v, see in seqs:
        n = see.shape[0]
        for h in range(Hq):
            x = q[t0:t0 + n, h]
            s = np.where(see, scale * (x @ k[h // group].T), -np.inf)
            mag = np.where(see, scale * (np.abs(x) @ np.abs(k[h // group]).T), 0.0)
            for i in np.nonzero(see.any(1))[0]:
                top = np.max(s[i])
                e = np.exp(s[i] - top)
                l = e.sum()
                o[t0 + i, h], av[t0 + i, h] = e @ v[h // group] / l, e @ np.abs(v[h // group]) / l
                lse[t0 + i, h], size[t0 + i, h] = top + math.log(l), np.max(mag[i])
    return o, lse, av, size


def compare(got_o, got_lse, want, dim, longest, dtype):
    """Asserts the bounds of serve_ref.paged_bounds (bf16: weights rounded to bf16), with eight fp32
    roundings more for results that are joined from two passes."""
    wo, wl, av, size = want
    to, tl = ref.paged_bounds(wo, wl, av, size, dim, longest, dtype, dtype == "bf16")
    to, tl = to + 8 * ref.F32 * av, tl + 8 * ref.F32 * (1 + np.abs(np.where(np.isfinite(wl), wl, 0.0)))
    assert got_o.shape == wo.shape and got_lse.shape == wl.shape
    assert not np.isnan(got_o).any() and not np.isnan(got_lse).any()
    fin = np.isfinite(wl)
    assert np.all(got_lse[~fin] == -np.inf)
    if fin.any():
        worst = np.max(np.abs(got_lse[fin] - wl[fin]) / tl[fin])
        assert worst <= 1, ("lse", float(worst))
    if wo.size:
        worst = np.abs(got_o - wo) / to
        assert np.max(worst) <= 1, (float(np.max(worst)), np.unravel_index(np.argmax(worst), worst.shape))


def poison_hidden(b, window, sinks):
    """Of a test_paged_gpu.Batch: what no query of a sequence sees becomes NaN (codes and scales too), and
    pages that hold nothing else leave the table.  The batch's own copies stay as they were."""
    import torch

    hidden = np.zeros((b.pages, b.page), bool)
    table = b.table_h.copy()
    for s in range(b.B):
        n, m = int(b.new[s]), int(b.lens_h[s])
        low = m if n == 0 else min(m, max(0, m - n - window + 1))
        for j in range(-(-m // b.page)):
            at = np.arange(j * b.page, (j + 1) * b.page)
            gone = (at >= sinks) & (at < low)
            if n == 0:
                gone = at >= 0
            hidden[table[s, j]] |= gone
            if gone.all():
                table[s, j] = -1 - j
    m = torch.tensor(hidden, device="cuda")[:, None, :, None]
    c = b.cache
    if c.mxfp8:
        for x in (c.k, c.v):
            x.copy_(torch.where(m, 0x7f, x.int()).to(torch.uint8))
        for x in (c.k_scale, c.v_scale):
            x.copy_(torch.where(m, 255, x.int()).to(torch.uint8))
    else:
        for x in (c.k, c.v):
            x.copy_(torch.where(m, torch.full_like(x, float("nan")), x))
    b.table.copy_(torch.tensor(table, dtype=torch.int32))
