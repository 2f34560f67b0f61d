"""Host-side refusals of windowed and shared attention over a paged cache: every check below returns before
a CUDA call is made."""
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


def G(**kw):
    base = dict(batch=2, total_q=5, pages=10, stride_q=256, stride_k=256, stride_v=256, heads_q=2, heads_k=2,
                dim_qk=128, dim_v=128, page_size=64, max_pages=4, scale=0.1, causal=1, dtype=jfa.JFA_BF16,
                cache_dtype=jfa.JFA_BF16, flags=0)
    base.update(kw)
    return jfa.jfa_paged_params(**base)


def ref(p):
    return ctypes.byref(p) if p is not None else None


def window(L, p, w=10, n=4, q=16, kc=16, ks=16, offs=16, lens=16, table=16, o=16, lse=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_paged_window_fwd(ref(p), w, n, vp(q), vp(kc), vp(kc), vp(ks), vp(ks), vp(offs), vp(lens), vp(table),
                                  vp(o), vp(lse), vp(ws), ws_bytes, None)


def plan(L, p, w=10, n=4, offs=16, lens=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_paged_window_plan(ref(p), w, n, vp(offs), vp(lens), vp(ws), ws_bytes, None)


def shared(L, p, groups=1, width=3, q=16, kc=16, ks=16, offs=16, lens=16, table=16, goffs=16, plens=16, ptable=16, o=16,
           lse=16, ws=256, ws_bytes=1 << 30):
    return L.jfa_shared_fwd(ref(p), groups, width, vp(q), vp(kc), vp(kc), vp(ks), vp(ks), vp(offs), vp(lens), vp(table),
                            vp(goffs), vp(plens), vp(ptable), vp(o), vp(lse), vp(ws), ws_bytes, None)


def test_common_refusals(L):
    for f in (window, plan, shared):
        assert f(L, None) == BAD
        for kw in (dict(batch=-1), dict(total_q=-1), dict(pages=-1), dict(heads_q=3), dict(dtype=2), dict(flags=2),
                   dict(scale=0.0), dict(scale=float("nan")), dict(causal=2), dict(page_size=0)):
            assert f(L, G(**kw)) == BAD, (f, kw)
        for kw in (dict(cache_dtype=jfa.JFA_F32), dict(page_size=8), dict(dim_qk=12), dict(dim_v=136),
                   dict(max_pages=1 << 26), dict(total_q=(1 << 31) - 255, batch=1)):
            assert f(L, G(**kw)) == UNSUP, (f, kw)
        assert f(L, G(), ws=0) == WS and f(L, G(), ws=128) == WS and f(L, G(), ws_bytes=256) == WS
        assert f(L, G(), offs=0) == BAD and f(L, G(), lens=4) == BAD
    for f in (window, shared):
        for kw in (dict(q=0), dict(q=8), dict(kc=0), dict(o=8), dict(lse=0), dict(table=2)):
            assert f(L, G(), **kw) == BAD, (f, kw)
        assert f(L, G(stride_q=255)) == BAD and f(L, G(stride_q=260)) == BAD
        assert f(L, G(cache_dtype=jfa.JFA_MXFP8), ks=0) == BAD


def test_window_refusals(L):
    for f in (window, plan):
        assert f(L, G(), w=0) == BAD and f(L, G(), w=-5) == BAD and f(L, G(), n=-1) == BAD
        assert f(L, G(causal=0)) == UNSUP


def test_shared_refusals(L):
    assert shared(L, G(), groups=-1) == BAD and shared(L, G(), groups=0) == BAD and shared(L, G(), width=-1) == BAD
    assert shared(L, G(), goffs=0) == BAD and shared(L, G(), plens=4) == BAD and shared(L, G(), ptable=2) == BAD
    assert shared(L, G(), width=1 << 26) == UNSUP and shared(L, G(), groups=1 << 31) == UNSUP
    assert shared(L, G(flags=jfa.JFA_PLANNED)) == UNSUP
    # costs past 64 bits: every row may see every position of the prefix
    assert shared(L, G(heads_q=65536, heads_k=1, total_q=(1 << 31) - 256, batch=1, max_pages=1), width=(1 << 25) - 4) == UNSUP
    size = lambda p, g, w: L.jfa_shared_workspace_size(ref(p), g, w)
    a = L.jfa_paged_workspace_size(ref(G()))
    rows = 5 * 2 * (128 + 1) * 4
    assert a + rows < size(G(), 1, 3) < a + rows + (1 << 16)
    assert size(None, 1, 3) == 0 and size(G(), -1, 3) == 0 and size(G(page_size=7), 1, 3) == 0
    assert shared(L, G(), ws_bytes=size(G(), 1, 3) - 1) == WS


def append(L, p, rope=None, norm=1, eps=1e-6, q=16, k=16, v=16, pos=16, wq=16, wk=16, offs=16, lens=16, table=16, yq=16,
           syq=256, kc=16, ks=16, ws=256, ws_bytes=1 << 30):
    rope = jfa.jfa_rope(128) if rope is None else rope
    return L.jfa_rope_append(ref(p), ctypes.byref(rope), norm, eps, vp(q), vp(k), vp(v), vp(pos), vp(wq), vp(wk), vp(offs),
                             vp(lens), vp(table), vp(yq), syq, vp(kc), vp(kc), vp(ks), vp(ks), vp(ws), ws_bytes, None)


def test_append_refusals(L):
    assert append(L, None) == BAD
    for kw in (dict(batch=-1), dict(total_q=-1), dict(pages=-1), dict(heads_q=0), dict(dtype=2), dict(flags=2),
               dict(stride_q=255), dict(stride_k=260), dict(stride_v=0)):
        assert append(L, G(**kw)) == BAD, kw
    for kw in (dict(cache_dtype=jfa.JFA_F32), dict(page_size=8), dict(dim_qk=12), dict(dim_v=264), dict(max_pages=1 << 26)):
        assert append(L, G(**kw)) == UNSUP, kw
    for kw in (dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=8), dict(k=0), dict(v=4), dict(pos=12), dict(wq=18),
               dict(offs=0), dict(lens=4), dict(table=2), dict(yq=0), dict(yq=8), dict(syq=255), dict(syq=260), dict(kc=0),
               dict(q=0), dict(norm=0), dict(rope=jfa.jfa_rope(130)), dict(rope=jfa.jfa_rope(64, base=0.5))):
        assert append(L, G(), **kw) == BAD, kw
    assert append(L, G(cache_dtype=jfa.JFA_MXFP8), ks=0) == BAD
    assert append(L, G(), ws=0) == WS and append(L, G(), ws=128) == WS and append(L, G(), ws_bytes=256) == WS


def P(**kw):
    base = dict(batch=2, total_q=10, total_k=10, heads=2, dim_qk=64, dim_v=64, scale=0.125, causal=1, dtype=jfa.JFA_BF16, flags=0)
    base.update(kw)
    return jfa.jfa_params(**base)


def train(L, p, w=10, n=4, ptr=16, offs=16, o=16, ws=256, ws_bytes=1 << 20):
    """Forward, backward and plan give the same answer."""
    got = {L.jfa_window_fwd(ref(p), w, n, vp(ptr), vp(ptr), vp(ptr), vp(offs), vp(o), vp(ptr), vp(ws), ws_bytes, None),
           L.jfa_window_bwd(ref(p), w, n, vp(ptr), vp(ptr), vp(ptr), vp(o), vp(ptr), vp(ptr), vp(offs), vp(ptr), vp(ptr),
                            vp(ptr), vp(ws), ws_bytes, None)}
    if ptr == 16 and o == 16:
        got.add(L.jfa_window_plan(ref(p), w, n, vp(offs), vp(ws), ws_bytes, None))
    assert len(got) == 1
    return got.pop()


def test_training_refusals(L):
    assert train(L, None) == BAD
    for kw in (dict(batch=-1), dict(total_q=-1), dict(total_k=9), dict(heads=0), dict(dim_v=0), dict(dtype=2),
               dict(scale=0.0), dict(causal=2), dict(flags=2)):
        assert train(L, P(**kw)) == BAD, kw
    for kw in (dict(causal=0), dict(dim_qk=129), dict(total_q=1 << 31, total_k=1 << 31)):
        assert train(L, P(**kw)) == UNSUP, kw
    for kw in (dict(w=0), dict(w=-1), dict(n=-1), dict(ptr=0), dict(ptr=8), dict(o=0), dict(offs=0)):
        assert train(L, P(), **kw) == BAD, kw
    assert train(L, P(), ws=0) == WS and train(L, P(), ws=128) == WS and train(L, P(), ws_bytes=1024) == WS
