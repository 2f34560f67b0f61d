"""Host-side refusals of the operators around attention over a paged cache: every check below
returns before a CUDA call is made."""
import ctypes

import pytest

import jagged_attention_recsys_gb300 as jfa
from jagged_attention_recsys_gb300 import build as jbuild

BAD, UNSUP, WS = jfa.JFA_ERR_INVALID_ARG, jfa.JFA_ERR_UNSUPPORTED, jfa.JFA_ERR_WORKSPACE
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    jbuild.build()
    return jfa.lib()


def N(rope=None, **kw):
    base = dict(tokens=5, stride_q=256, stride_k=256, stride_yq=256, stride_yk=256, stride_dq=256, stride_dk=256,
                heads_q=2, heads_k=2, dim=128, dtype=jfa.JFA_BF16, norm=1, eps=1e-6)
    base.update(kw)
    p = jfa.jfa_norm_rope_params(**base)
    p.rope = jfa.jfa_rope(128) if rope is None else rope
    return p


def fwd(L, p, q=16, k=16, pos=16, wq=16, wk=16, yq=16, yk=16):
    return L.jfa_norm_rope_fwd(ctypes.byref(p) if p is not None else None, vp(q), vp(k), vp(pos), vp(wq), vp(wk),
                               vp(yq), vp(yk), None)


def bwd(L, p, dyq=16, dq=16, ws=256, ws_bytes=1 << 24, norm_w=16):
    return L.jfa_norm_rope_bwd(ctypes.byref(p), vp(16), vp(16), vp(16), vp(norm_w), vp(norm_w), vp(dyq), vp(16),
                               vp(dq), vp(16), vp(norm_w), vp(norm_w), vp(ws), ws_bytes, None)


def test_norm_rope_refusals(L):
    assert fwd(L, None) == BAD
    for kw in (dict(tokens=-1), dict(heads_q=-1), dict(heads_q=0, heads_k=0), dict(dim=0), dict(dtype=2), dict(norm=2),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(stride_q=255), dict(stride_yk=0),
               dict(stride_q=-256)):
        assert fwd(L, N(**kw)) == BAD, kw
    for kw in (dict(dim=257), dict(tokens=1 << 31), dict(heads_q=65536)):
        assert fwd(L, N(**kw)) == UNSUP, kw
    r = jfa.jfa_rope
    inf, nan = float("inf"), float("nan")
    for rope in (r(130), r(127), r(-2), r(64, base=0.5), r(64, base=nan), r(64, amp=inf),
                 r(64, scaling="linear", factor=0.5), r(64, scaling="ntk", factor=nan), r(2, scaling="ntk", factor=2.0),
                 r(64, scaling="yarn", factor=2.0), r(64, scaling="yarn", factor=2.0, orig_len=100, turns_fast=1.0),
                 r(64, scaling="yarn", factor=2.0, orig_len=inf),
                 r(64, scaling="yarn", factor=2.0, orig_len=100, turns_slow=-1.0)):
        assert fwd(L, N(rope)) == BAD
    bad = r(64)
    bad.layout = 2
    assert fwd(L, N(bad)) == BAD
    bad = r(64)
    bad.scaling = 9
    assert fwd(L, N(bad)) == BAD
    p = N()
    assert fwd(L, p, q=0) == BAD and fwd(L, p, k=17) == BAD and fwd(L, p, pos=0) == BAD and fwd(L, p, pos=12) == BAD
    assert fwd(L, p, wq=18) == BAD and fwd(L, p, yq=0) == BAD
    assert fwd(L, N(dtype=jfa.JFA_F32), q=18) == BAD
    assert fwd(L, N(norm=0)) == BAD  # weights without a norm
    assert bwd(L, p, dyq=0) == BAD and bwd(L, p, dq=0) == BAD
    assert bwd(L, p, ws=0) == WS and bwd(L, p, ws=128) == WS and bwd(L, p, ws_bytes=1024) == WS
    assert bwd(L, N(norm=0)) == BAD
    assert L.jfa_norm_rope_workspace_size(ctypes.byref(p)) > 0
    assert L.jfa_norm_rope_workspace_size(ctypes.byref(N(dim=0))) == 0
    assert L.jfa_norm_rope_workspace_size(None) == 0
    assert fwd(L, N(tokens=0), q=0, k=0, pos=0, yq=0, yk=0) == jfa.JFA_OK


def G(**kw):
    base = dict(batch=2, total_q=5, pages=10, stride_q=256, stride_k=256, stride_v=256, heads_q=2, heads_k=2,
                dim_qk=128, dim_v=128, page_size=64, max_pages=4, scale=0.1, causal=1, dtype=jfa.JFA_BF16,
                cache_dtype=jfa.JFA_BF16, flags=0)
    base.update(kw)
    return jfa.jfa_paged_params(**base)


def paged(L, p, q=16, kc=16, ks=16, offs=16, lens=16, table=16, o=16, lse=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_paged_fwd(ctypes.byref(p) if p is not None else None, vp(q), vp(kc), vp(kc), vp(ks), vp(ks), vp(offs),
                           vp(lens), vp(table), vp(o), vp(lse), vp(ws), ws_bytes, None)


def write(L, p, k=16, kc=16, ks=16, offs=16, lens=16, table=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_cache_write(ctypes.byref(p), vp(k), vp(k), vp(offs), vp(lens), vp(table), vp(kc), vp(kc), vp(ks),
                             vp(ks), vp(ws), ws_bytes, None)


def read(L, p, k=16, kc=16, ks=16, offs=16, lens=16, table=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_cache_read(ctypes.byref(p), vp(kc), vp(kc), vp(ks), vp(ks), vp(offs), vp(lens), vp(table), vp(k),
                            vp(k), vp(ws), ws_bytes, None)


def plan(L, p, offs=16, lens=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_paged_plan(ctypes.byref(p), vp(offs), vp(lens), vp(ws), ws_bytes, None)


def test_paged_refusals(L):
    every = (paged, write, read, plan)
    assert paged(L, None) == BAD
    for kw in (dict(batch=-1), dict(total_q=-1), dict(pages=-1), dict(heads_k=0), dict(heads_q=0), dict(dim_qk=0),
               dict(max_pages=-1), dict(batch=0), dict(dtype=2), dict(cache_dtype=3), dict(flags=2),
               dict(page_size=0)):
        for f in every:
            assert f(L, G(**kw)) == BAD, (kw, f)
    for kw in (dict(cache_dtype=jfa.JFA_F32), dict(page_size=8), dict(page_size=48), dict(page_size=512),
               dict(dim_qk=12), dict(dim_v=264), dict(cache_dtype=jfa.JFA_MXFP8, dim_qk=48),
               dict(total_q=1 << 31, batch=1), dict(batch=1 << 31), dict(pages=1 << 31), dict(max_pages=1 << 26),
               dict(heads_q=1 << 17, heads_k=1 << 17)):
        for f in every:
            assert f(L, G(**kw)) == UNSUP, (kw, f)
    for kw in (dict(heads_q=3), dict(causal=2), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        for f in (paged, plan):
            assert f(L, G(**kw)) == BAD, (kw, f)
    assert paged(L, G(dim_qk=136)) == UNSUP and plan(L, G(dim_v=136)) == UNSUP
    # costs past 64 bits
    assert plan(L, G(heads_q=65536, heads_k=1, total_q=(1 << 31) - 1, batch=1, max_pages=(1 << 25) - 1)) == UNSUP
    for f in every:
        assert f(L, G(), offs=0) == BAD and f(L, G(), lens=4) == BAD
        assert f(L, G(), ws=0) == WS and f(L, G(), ws=128) == WS and f(L, G(), ws_bytes=256) == WS
    for f in (paged, write, read):
        assert f(L, G(), table=2) == BAD and f(L, G(), kc=0) == BAD and f(L, G(), kc=24) == BAD
        assert f(L, G(cache_dtype=jfa.JFA_MXFP8), ks=0) == BAD
    assert paged(L, G(), q=0) == BAD and paged(L, G(), q=8) == BAD and paged(L, G(), o=0) == BAD
    assert paged(L, G(), lse=8) == BAD
    assert paged(L, G(stride_q=255)) == BAD and paged(L, G(stride_q=260)) == BAD
    assert write(L, G(), k=0) == BAD and write(L, G(stride_k=0)) == BAD and write(L, G(stride_v=257)) == BAD
    assert read(L, G(), k=8) == BAD
    a = L.jfa_paged_workspace_size(ctypes.byref(G()))
    assert 0 < a <= 64 << 20
    assert L.jfa_paged_workspace_size(ctypes.byref(G(batch=1 << 20))) > a
    assert L.jfa_paged_workspace_size(ctypes.byref(G(page_size=7))) == 0
    assert L.jfa_paged_workspace_size(None) == 0


def test_positions_that_tiles_would_carry_past_32_bits(L):
    """A tile's end is worked out in 32 bits: the last 255 values are refused."""
    for f in (paged, write, read, plan):
        assert f(L, G(page_size=16, max_pages=(1 << 27) - 15)) == UNSUP
        assert f(L, G(total_q=(1 << 31) - 255, batch=1)) == UNSUP
    assert L.jfa_paged_workspace_size(ctypes.byref(G(page_size=16, max_pages=(1 << 27) - 16, total_q=(1 << 31) - 256))) > 0


def test_status_names_bad_pages(L):
    assert "page" in jfa.status_string(jfa.JFA_ERR_BAD_PAGES)
