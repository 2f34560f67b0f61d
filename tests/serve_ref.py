"""Plain 64-bit implementations of the operators around attention over a paged cache (norms with
rotary positions, the MXFP8 cache, the attention), for the tests, with the error bounds that the
types of the kernels allow.  numpy and the pinned MXFP8 oracle only."""
from __future__ import annotations

import math

import numpy as np

from oracle import mxfp8

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of a stored value, relative
F32 = 2.0 ** -24


# ------------------------------------------------------------------ norms and rotary positions
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, turns_fast=32.0, turns_slow=1.0):
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2.0)) if scaling == "ntk" else base
        t = b ** (-2.0 * i / rot)
        if scaling == "linear":
            t = t / factor
        if scaling == "yarn":
            g = (orig_len * t / (2 * math.pi) - turns_slow) / (turns_fast - turns_slow)
            g = min(1.0, max(0.0, g))
            t = t * (g + (1.0 - g) / factor)
        out.append(t)
    return np.array(out, dtype=np.float64)


def pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "halves" else (2 * i, 2 * i + 1)


def _turn(x, pos, freq, rot, layout, amp, sign):
    y = x.copy()
    if rot:
        ang = pos.astype(np.float64)[:, None] * freq
        c, s = (amp * np.cos(ang))[:, None], (sign * amp * np.sin(ang))[:, None]
        a, b = pairs(rot, layout)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _reach(x, rot, layout, amp):
    """Of every column: the size of what it is computed from (a pair's length)."""
    y = np.abs(x)
    if rot:
        a, b = pairs(rot, layout)
        h = abs(amp) * np.hypot(x[..., a], x[..., b])
        y[..., a], y[..., b] = h, h
    return y


def norm_rope(x, w, pos, freq, rot, layout, amp, eps, norm=True):
    """(y, size of what each value is computed from); x [T, H, D] in 64 bits."""
    n = x
    if norm:
        n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * (1.0 if w is None else w)
    return _turn(n, pos, freq, rot, layout, amp, 1.0), _reach(n, rot, layout, amp)


def norm_rope_bwd(x, w, pos, freq, rot, layout, amp, eps, dy, norm=True):
    """(dx, dw, size for dx, size for dw)."""
    g = _turn(dy, pos, freq, rot, layout, amp, -1.0)
    gr = _reach(dy, rot, layout, amp)
    if not norm:
        return g, None, gr, None
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    ww = 1.0 if w is None else w
    u, ur = g * ww, gr * np.abs(ww)
    dx = r * (u - x * r * r * np.mean(u * x, -1, keepdims=True))
    size = r * (ur + np.abs(x) * r * r * np.mean(ur * np.abs(x), -1, keepdims=True))
    return dx, np.sum(g * x * r, (0, 1)), size, np.sum(gr * np.abs(x) * r, (0, 1))


# ------------------------------------------------------------------------------------ the cache
def quantize_rows(x):
    """(codes' values times scale, values of the codes alone, exponents) of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    nb = flat.shape[1] // 32
    e = np.empty((flat.shape[0], nb), np.int64)
    code = np.empty_like(flat)
    for c in range(nb):
        blk = flat[:, 32 * c:32 * c + 32]
        e[:, c] = np.clip(mxfp8.block_scale_exp(np.max(np.abs(blk), axis=1)), -100, 119)
        code[:, 32 * c:32 * c + 32] = mxfp8.e4m3_quantize(blk / np.ldexp(1.0, e[:, c])[:, None])
    val = code * np.repeat(np.ldexp(1.0, e), 32, axis=1)
    return val.reshape(x.shape), code.reshape(x.shape), e.reshape(x.shape[:-1] + (nb,))


_DECODE = np.array([mxfp8.e4m3_decode(c) for c in range(256)])


def decode(codes, scales):
    """Values of uint8 codes [..., D] with biased exponents [..., D / 32]."""
    return _DECODE[codes] * np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32, axis=-1)


def rows_of(cache, table, b, n):
    """The first n positions of sequence b: cache [pages, heads, page, D] -> [heads, n, D]."""
    ps = cache.shape[2]
    pages = [int(table[b, j]) for j in range(-(-n // ps))]
    if not pages:
        return np.zeros((cache.shape[1], 0, cache.shape[3]), cache.dtype)
    return np.concatenate([cache[p] for p in pages], axis=1)[:, :n]


# ------------------------------------------------------------------------------- the attention
def paged(q, k_of, v_of, offs, lens, group, scale, causal):
    """q [T, Hq, D]; k_of(b), v_of(b): [Hk, lens[b], D].  Returns o, lse and, for the bounds,
    sum_j p_j |v_j| and the largest scale * sum_d |q_d k_jd| of every row."""
    T, Hq, _ = q.shape
    B = len(offs) - 1
    Dv = v_of(0).shape[2] if B else 0
    o, av = np.zeros((T, Hq, Dv)), np.zeros((T, Hq, Dv))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(B):
        k, v, L = k_of(b), v_of(b), int(lens[b])
        n = int(offs[b + 1] - offs[b])
        for h in range(Hq):
            x = q[offs[b]:offs[b + 1], h]
            s = scale * (x @ k[h // group].T)
            mag = scale * (np.abs(x) @ np.abs(k[h // group]).T)
            for i in range(n):
                m = min(L, max(0, L - n + i + 1)) if causal else L
                if m == 0:
                    continue
                t = int(offs[b]) + i
                top = np.max(s[i, :m])
                e = np.exp(s[i, :m] - top)
                l = e.sum()
                o[t, h] = e @ v[h // group][:m] / l
                av[t, h] = e @ np.abs(v[h // group][:m]) / l
                lse[t, h] = top + math.log(l)
                size[t, h] = np.max(mag[i, :m])
    return o, lse, av, size


def paged_bounds(o, lse, av, size, dim, longest, out, rounded_weights):
    """Largest errors of o and lse.  A score is a sum of `dim` products in fp32 (each step within
    2 units of 2^-24, as tensor cores may cut where they do not round), scaled and moved by the
    maximum (4 more roundings of at most its size); a weight's relative error is then the
    score's absolute error plus that of exp2 (2^-22); sums over up to `longest` keys in fp32
    add 2 longest units at most along one chain, of which the kernels make chains no longer
    than 256 before partial sums meet.  Weights rounded to bf16 add 2^-8 of sum p |v|.  The
    result is rounded once to its type."""
    ds = 2 * F32 * (dim + 8) * size + 8 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 2.0 ** -22
    rel = 2 * ds + 2 * F32 * min(longest, 512) + (2.0 ** -8 if rounded_weights else 0.0)
    tol_o = rel[..., None] * av + HALF_STEP[out] * np.abs(o) * 1.01 + 1e-30
    tol_l = ds + 2 * F32 * min(longest, 512) + 4 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol_o, tol_l
