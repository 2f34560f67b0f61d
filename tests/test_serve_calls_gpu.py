"""The calls around attention over a paged cache as a program makes them: refused arguments,
other streams, batches at the size from which the work is planned in a launch of its own, and
plans that no longer fit.  GPU only."""
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
from test_paged_gpu import Batch, _poisoned, check_attention

pytestmark = pytest.mark.gpu


def small(cache="bf16"):
    b = Batch([2, 3], [40, 20], 2, 64, 64, 16, cache, "bf16")
    q = torch.randn(5, 4, 64, device="cuda").bfloat16()
    k, v = (torch.randn(5, 2, 64, device="cuda").bfloat16() for _ in range(2))
    return b, q, k, v


def test_refused_caches():
    z = lambda *s, t=torch.bfloat16, d="cuda": torch.zeros(*s, dtype=t, device=d)
    u = torch.uint8
    for bad in (lambda: jfa.PagedCache(z(4, 2, 16, 64), z(3, 2, 16, 64)),
                lambda: jfa.PagedCache(z(4, 2, 16), z(4, 2, 16)),
                lambda: jfa.PagedCache(z(4, 2, 16, 64), z(4, 2, 16, 64, t=torch.float32)),
                lambda: jfa.PagedCache(z(4, 2, 16, 64, d="cpu"), z(4, 2, 16, 64, d="cpu")),
                lambda: jfa.PagedCache(z(4, 2, 64, 16).transpose(2, 3), z(4, 2, 16, 64)),
                lambda: jfa.PagedCache(z(4, 2, 16, 64, t=u), z(4, 2, 16, 64, t=u), z(4, 2, 16, 2, t=u)),
                lambda: jfa.PagedCache(z(4, 2, 16, 64, t=u), z(4, 2, 16, 64, t=u), z(4, 2, 16, 4, t=u), z(4, 2, 16, 2, t=u)),
                lambda: jfa.PagedCache(z(4, 2, 16, 64), z(4, 2, 16, 64), z(4, 2, 16, 2, t=u), z(4, 2, 16, 2, t=u)),
                lambda: jfa.PagedCache(z(4, 2, 16, 48, t=u), z(4, 2, 16, 64, t=u), z(4, 2, 16, 1, t=u), z(4, 2, 16, 2, t=u))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        jfa.PagedCache(z(4, 2, 16, 64, t=torch.float16), z(4, 2, 16, 64, t=torch.float16))


def test_refused_calls_leave_the_outputs():
    b, q, k, v = small()
    o, lse = _poisoned(b, 4)
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, 5, torch.bfloat16, heads_q=4))
    t, f, n = b.table, b.offs, b.lens
    fwd, write, read, plan = jfa.jfa_paged_fwd, jfa.jfa_cache_write, jfa.jfa_cache_read, jfa.jfa_paged_plan
    for bad in (lambda: fwd(q, b.cache, t.long(), f, n), lambda: fwd(q, b.cache, t, f.int(), n),
                lambda: fwd(q, b.cache, t, f, n[:1]), lambda: fwd(q, b.cache, t[:1], f, n),
                lambda: fwd(q, b.cache, t.t(), f, n), lambda: fwd(q, b.cache, t, f.cpu(), n),
                lambda: fwd(q, b.cache, t[0], f, n), lambda: fwd(q, b.cache, t, f[:0], n),
                lambda: fwd(q[0], b.cache, t, f, n), lambda: fwd(q[0, 0], b.cache, t, f, n),
                lambda: fwd(q[:, :, :32], b.cache, t, f, n), lambda: fwd(q.cpu(), b.cache, t, f, n),
                lambda: fwd(q, b.cache, t, f, n, o=o.float()), lambda: fwd(q, b.cache, t, f, n, o=o[:4]),
                lambda: fwd(q, b.cache, t, f, n, lse=lse.t()), lambda: fwd(q, b.cache, t, f, n, lse=lse.double()),
                lambda: fwd(q, b.cache, t, f, n, planned=True), lambda: fwd(q, b.cache, t, f, n, ws=ws.float()),
                lambda: fwd(q, b.cache, t, f, n, ws=ws.cpu()), lambda: fwd(q, b.cache, t, f, n, ws=ws[::2]),
                lambda: write(k[:4], v, b.cache, t, f, n), lambda: write(k, v.float(), b.cache, t, f, n),
                lambda: write(k[:, :1], v, b.cache, t, f, n), lambda: write(k, v.transpose(1, 2), b.cache, t, f, n),
                lambda: read(b.cache, t, f, n, 5, k=k.float()), lambda: read(b.cache, t, f, n, 4, k=k),
                lambda: plan(q[0], b.cache, t, f, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fwd(q.half(), b.cache, t, f, n)
    for bad in (lambda: fwd(q.float(), b.cache, t, f, n),                 # a cache of another type
                lambda: fwd(q[:, :3].contiguous(), b.cache, t, f, n),     # heads that do not divide
                lambda: fwd(q, b.cache, t, f, n, ws=ws[:256]), lambda: fwd(q, b.cache, t, f, n, ws=ws[16:]),
                lambda: fwd(q, b.cache, t, f, n, scale=0.0), lambda: read(b.cache, t, f, n, 5, dtype=torch.float32),
                lambda: fwd(q[:1].expand(5, 4, 64), b.cache, t, f, n),    # tokens that share memory
                lambda: write(k, v, jfa.PagedCache(b.cache.k[:, :, :8].contiguous(), b.cache.v[:, :, :8].contiguous()), t, f, n)):
        with pytest.raises(jfa.JfaError):
            bad()
    torch.cuda.synchronize()
    assert bool((o == 3).all()) and bool((lse == 3).all())


def test_calls_on_a_stream_of_their_own():
    """What a call allocates belongs to the stream it runs on: later allocations of the current
    stream do not get its memory while it runs."""
    b, q, k, v = small("mxfp8")
    want, wl = jfa.jfa_paged_fwd(q, *b.args())
    rk, rv = jfa.jfa_cache_read(*b.args(), 5)
    x = torch.randn(300, 4, 64, device="cuda").bfloat16()
    pos, w = torch.arange(300, device="cuda"), torch.rand(64, device="cuda")
    rope = jfa.jfa_rope(64)
    y = jfa.jfa_norm_rope_fwd(x, x, pos, w, w, rope=rope)
    g = jfa.jfa_norm_rope_bwd(x, x, pos, x, x, w, w, rope=rope)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = jfa.jfa_paged_fwd(q, *b.args(), stream=s)
        gk, gv = jfa.jfa_cache_read(*b.args(), 5, stream=s)
        ws = jfa.jfa_paged_plan(q, *b.args(), stream=s)
        planned = jfa.jfa_paged_fwd(q, *b.args(), ws=ws, planned=True, stream=s)
        y2 = jfa.jfa_norm_rope_fwd(x, x, pos, w, w, rope=rope, stream=s)
        g2 = jfa.jfa_norm_rope_bwd(x, x, pos, x, x, w, w, rope=rope, stream=s)
        [torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert torch.cuda.current_stream() != s
        s.synchronize()
        for a, e in zip((*got, *planned, gk, gv, *y2, *g2), (want, wl, want, wl, rk, rv, *y, *g)):
            assert torch.equal(a, e)
    before = b.cache.k.clone()
    jfa.jfa_cache_write(k, v, *b.args(), stream=s)
    s.synchronize()
    assert not torch.equal(before, b.cache.k)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "mxfp8")])
@pytest.mark.parametrize("B", [1, 31, 127, 128, 129, 511, 512, 513])
def test_batches_around_the_size_that_is_planned_apart(B, dtype, cache):
    """The shares are the same whoever cuts them, so the results are, bit for bit; sequences without
    tokens or keys among them."""
    new = [(7 * i) % 3 for i in range(B)]
    lens = [(13 * i) % 61 + (400 if i == B - 1 else 0) for i in range(B)]
    b = Batch(new, lens, 2, 64, 64, 16, cache, dtype)
    if b.T == 0:
        b = Batch([2] * B, lens, 2, 64, 64, 16, cache, dtype)
    q, o, lse = check_attention(b, 4)
    ws = jfa.jfa_paged_plan(q, *b.args())
    o2, lse2 = jfa.jfa_paged_fwd(q, *b.args(), ws=ws, planned=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    # an unplanned call leaves a plan in its workspace too
    ws.fill_(0xa5)
    jfa.jfa_paged_fwd(q, *b.args(), ws=ws)
    o3, lse3 = jfa.jfa_paged_fwd(q, *b.args(), ws=ws, planned=True)
    assert torch.equal(o, o3) and torch.equal(lse, lse3) and jfa.jfa_status_check(ws) == jfa.JFA_OK


@pytest.mark.parametrize("B", [128, 512, 513])
@pytest.mark.parametrize("at", ["first", "last", "inside"])
def test_invalid_batches_of_many_sequences(B, at):
    b = Batch([1] * B, [20] * B, 1, 64, 64, 16, "bf16", "bf16")
    b.lens[{"first": 0, "last": B - 1, "inside": B // 2}[at]] = -5
    o, lse = _poisoned(b, 8)
    q = torch.randn(B, 8, 64, device="cuda").bfloat16()
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, B, torch.bfloat16, heads_q=8))
    jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
    assert bool((o == 3).all()) and bool((lse == 3).all())
    # and the next call on the workspace starts afresh
    b.lens.fill_(20)
    check_attention(b, 8, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK


def test_weight_gradients_of_a_tensor_without_heads_are_zero():
    k = torch.randn(30, 2, 64, device="cuda")
    pos, w = torch.arange(30, device="cuda"), torch.rand(64, device="cuda")
    none = k[:, :0]
    dwq = torch.full((64,), 7.0, device="cuda")
    _, dk, got, dwk = jfa.jfa_norm_rope_bwd(none, k, pos, none, k, w, w, rope=jfa.jfa_rope(64), dwq=dwq)
    assert got is dwq and bool((dwq == 0).all())
    _, dk2, _, dwk2 = jfa.jfa_norm_rope_bwd(None, k, pos, None, k, None, w, rope=jfa.jfa_rope(64))
    assert torch.equal(dk, dk2) and torch.equal(dwk, dwk2) and bool((dwk != 0).any())
