"""The paged cache (jfa_cache_write / jfa_cache_read) and attention over it (jfa_paged_plan /
jfa_paged_fwd) against plain 64-bit implementations.  GPU only.

Slots that no sequence owns, pages that no table names and table entries behind a sequence's
pages hold NaN or nonsense throughout: none of it may reach a result."""
import ctypes

import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """A cache with everything unowned poisoned, and its sequences' rows."""

    def __init__(self, new, lens, hk, dqk, dv, page, cache, dtype, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.new, self.lens_h = np.array(new, np.int64), np.array(lens, np.int64)
        self.offs_h = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)
        self.B, self.T, self.page, self.hk = len(new), int(self.offs_h[-1]), page, hk
        used = [-(-int(n) // page) for n in lens]
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages)
        width = max(used + [1]) + 1
        # entries behind a sequence's pages are nonsense
        self.table_h = rng.choice(np.array([-1, self.pages, 2 ** 31 - 1, -2 ** 31], np.int64), (self.B, width))
        at = 0
        for b, n in enumerate(used):
            self.table_h[b, :n] = order[at:at + n]
            at += n
        self.dtype, self.kind, self.dqk, self.dv = dtype, cache, dqk, dv
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = lambda a, t: torch.tensor(a, dtype=t, device="cuda")
        self.offs, self.lens = dev(self.offs_h, torch.int64), dev(self.lens_h, torch.int64)
        self.table = dev(self.table_h, torch.int32)
        owned = torch.zeros(self.pages, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(used):
            for j in range(n):
                owned[self.table_h[b, j], :min(page, int(lens[b]) - j * page)] = True
        self.owned = owned[:, None, :, None]
        shape = lambda d: (self.pages, hk, page, d)
        if cache == "mxfp8":
            arr = []
            for d in (dqk, dv):
                # any finite code; scales around 1 with a wide spread
                c = torch.randint(0, 256, shape(d), generator=g, device="cuda", dtype=torch.int32)
                c = torch.where((c & 127) == 127, c - 1, c)
                s = torch.randint(116, 122, shape(d // 32), generator=g, device="cuda", dtype=torch.int32)
                arr += [torch.where(self.owned, c, 0x7f).to(torch.uint8), torch.where(self.owned, s, 255).to(torch.uint8)]
            self.cache = jfa.PagedCache(arr[0], arr[2], arr[1], arr[3])
            self.k_h, self.v_h = (ref.decode(a.cpu().numpy(), s.cpu().numpy()) for a, s in ((arr[0], arr[1]), (arr[2], arr[3])))
        else:
            k, v = (torch.randn(shape(d), generator=g, device="cuda") for d in (dqk, dv))
            nan = torch.tensor(float("nan"), device="cuda")
            k, v = (torch.where(self.owned, x, nan).to(DT[dtype]) for x in (k, v))
            self.cache = jfa.PagedCache(k, v)
            self.k_h, self.v_h = f64(k), f64(v)

    def k_of(self, b):
        return ref.rows_of(self.k_h, self.table_h, b, int(self.lens_h[b]))

    def v_of(self, b):
        return ref.rows_of(self.v_h, self.table_h, b, int(self.lens_h[b]))

    def args(self):
        return self.cache, self.table, self.offs, self.lens


def rounded_weights(b, hq):
    """Whether the tensor-core kernels serve the request (they round the weights to bf16)."""
    return b.dtype == "bf16"


def check_attention(b, hq, causal=True, scale=None, seed=1, q=None, o=None, lse=None, **kw):
    if q is None:
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn(b.T, hq, b.dqk, generator=g, device="cuda").to(DT[b.dtype])
    o, lse = jfa.jfa_paged_fwd(q, *b.args(), causal=causal, scale=scale, o=o, lse=lse, **kw)
    assert o.shape == (b.T, hq, b.dv) and lse.shape == (b.T, hq)
    if b.T == 0:
        return q, o, lse
    s = b.dqk ** -0.5 if scale is None else scale
    wo, wl, av, size = ref.paged(f64(q), b.k_of, b.v_of, b.offs_h, b.lens_h, hq // b.hk, float(np.float32(s)), causal)
    to, tl = ref.paged_bounds(wo, wl, av, size, b.dqk, int(b.lens_h.max(initial=1)), b.dtype, rounded_weights(b, hq))
    go, gl = f64(o), f64(lse)
    assert np.array_equal(np.isfinite(wl), np.isfinite(gl)) and not np.isnan(gl).any()
    fin = np.isfinite(wl)
    if fin.any():
        assert np.max(np.abs(gl[fin] - wl[fin]) / tl[fin]) <= 1
    assert np.all(gl[~fin] == -np.inf)
    assert not np.isnan(go).any()
    worst = np.abs(go - wo) / to
    assert worst.size == 0 or np.max(worst) <= 1, (float(np.max(worst)), np.unravel_index(np.argmax(worst), worst.shape))
    return q, o, lse


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300, 700]


def ragged(kind):
    """(new, lens) of a batch."""
    rng = np.random.default_rng(7)
    if kind == "step":  # one token each, lengths at the edges (an empty sequence has no token)
        return [1 if n else 0 for n in EDGES], EDGES
    if kind == "prompt":  # whole prompts
        return EDGES, EDGES
    if kind == "chunk":  # some cached, some new; more new tokens than cached positions too
        new = [0, 1, 3, 16, 2, 40, 64, 5, 127, 130, 9, 257, 20, 300, 33]
        return new, [max(0, n + d) for n, d in zip(new, [5, 0, 40, 0, -1, 100, 64, -5, 1, 200, 500, 0, 900, -100, 128])]
    if kind == "one long":
        return [1], [5000]
    if kind == "one long chunk":
        return [70], [3000]
    if kind == "many short":
        lens = rng.integers(1, 40, 700)
        return np.minimum(lens, rng.integers(1, 3, 700)).tolist(), lens.tolist()
    if kind == "mixed":  # a prompt among single tokens
        return [1] * 20 + [400] + [1] * 20, [int(x) for x in rng.integers(1, 600, 20)] + [450] + [30] * 20
    raise KeyError(kind)


CASES = [
    # kind, dtype, cache, hq, hk, dqk, dv, page, causal
    ("step", "f32", "f32", 4, 2, 64, 64, 16, True),
    ("chunk", "f32", "f32", 3, 1, 40, 24, 32, True),
    ("chunk", "f32", "mxfp8", 4, 4, 32, 96, 16, False),
    ("prompt", "f32", "f32", 2, 2, 128, 128, 64, True),
    ("one long", "f32", "mxfp8", 8, 2, 128, 128, 256, True),
    ("chunk", "bf16", "bf16", 4, 2, 72, 8, 16, True),
    ("step", "bf16", "bf16", 8, 8, 64, 64, 16, True),
    ("step", "bf16", "bf16", 8, 1, 128, 128, 64, True),
    ("step", "bf16", "mxfp8", 32, 4, 128, 128, 32, True),
    ("step", "bf16", "mxfp8", 3, 1, 64, 64, 128, True),
    ("step", "bf16", "mxfp8", 14, 2, 128, 64, 64, False),
    ("step", "bf16", "bf16", 20, 1, 64, 128, 256, True),
    ("step", "bf16", "bf16", 48, 2, 128, 128, 16, True),
    ("chunk", "bf16", "bf16", 4, 4, 128, 128, 64, True),
    ("chunk", "bf16", "bf16", 8, 1, 64, 64, 16, True),
    ("chunk", "bf16", "bf16", 14, 2, 128, 64, 128, False),
    ("chunk", "bf16", "mxfp8", 4, 1, 128, 128, 32, True),
    ("chunk", "bf16", "mxfp8", 9, 3, 64, 128, 64, True),
    ("chunk", "bf16", "mxfp8", 40, 1, 128, 128, 16, True),
    ("prompt", "bf16", "bf16", 2, 2, 128, 128, 128, True),
    ("prompt", "bf16", "bf16", 8, 1, 64, 64, 256, True),
    ("prompt", "bf16", "mxfp8", 6, 2, 128, 128, 64, True),
    ("one long", "bf16", "bf16", 8, 1, 128, 128, 64, True),
    ("one long", "bf16", "mxfp8", 4, 2, 64, 64, 32, True),
    ("one long chunk", "bf16", "bf16", 8, 2, 128, 128, 64, True),
    ("one long chunk", "bf16", "mxfp8", 8, 1, 128, 128, 16, True),
    ("many short", "bf16", "bf16", 4, 4, 64, 64, 16, True),
    ("many short", "bf16", "mxfp8", 8, 2, 128, 128, 16, True),
    ("mixed", "bf16", "bf16", 8, 2, 128, 128, 64, True),
    ("mixed", "bf16", "mxfp8", 4, 4, 64, 64, 32, False),
    ("chunk", "bf16", "bf16", 130, 1, 64, 64, 64, True),
]


@pytest.mark.parametrize("case", CASES, ids=["%s-%s-%s-%d-%d-D%d-%d-p%d-%d" % c for c in CASES])
def test_attention(case):
    kind, dtype, cache, hq, hk, dqk, dv, page, causal = case
    b = Batch(*ragged(kind), hk, dqk, dv, page, cache, dtype)
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, DT[dtype], heads_q=hq))
    q, o, lse = check_attention(b, hq, causal, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    # the same bits again, and on work cut beforehand
    o2, lse2 = jfa.jfa_paged_fwd(q, *b.args(), causal=causal)
    ws = jfa.jfa_paged_plan(q, *b.args(), causal=causal)
    o3, lse3 = jfa.jfa_paged_fwd(q, *b.args(), causal=causal, ws=ws, planned=True)
    o4, lse4 = jfa.jfa_paged_fwd(q, *b.args(), causal=causal, ws=ws, planned=True)
    for a, l in ((o2, lse2), (o3, lse3), (o4, lse4)):
        assert torch.equal(a, o) and torch.equal(l, lse)


def test_large_scores_and_scale():
    """Scores of some hundreds: the running maximum moves often and most weights underflow."""
    for kind, new in (("step", 1), ("prompt", None)):
        n, lens = ragged(kind)
        b = Batch(n, lens, 2, 128, 128, 32, "bf16", "bf16", seed=4)
        check_attention(b, 4, scale=3.0)


@pytest.mark.parametrize("low,high", [(119, 136), (60, 190), (1, 3), (223, 230)])
@pytest.mark.parametrize("kind,hq,hk,dqk,dv", [("step", 8, 2, 128, 128), ("chunk", 3, 1, 64, 64), ("chunk", 8, 2, 128, 64),
                                               ("one long", 4, 2, 64, 128)])
def test_mxfp8_values_of_any_size(kind, hq, hk, dqk, dv, low, high):
    """Values whose scales lie up to the whole range apart, key by key and block by block: every
    column keeps its precision relative to its own sum of p |v|."""
    b = Batch(*ragged(kind), hk, dqk, dv, 32, "mxfp8", "bf16", seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    s = torch.randint(low, high + 1, b.cache.v_scale.shape, generator=g, device="cuda", dtype=torch.int32)
    # some blocks of columns only, and some keys
    s = torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.5, s, (low + high) // 2)
    b.cache.v_scale.copy_(torch.where(b.owned, s, 255).to(torch.uint8))
    v, vs = b.cache.v.cpu().numpy(), b.cache.v_scale.cpu().numpy()
    b.v_h = ref.decode(v, vs)
    check_attention(b, hq)


def test_rows_behind_the_last_and_strided_queries():
    """Queries as a slice of a projection's output; rows behind the call's stay as they were."""
    n, lens = ragged("chunk")
    b = Batch(n, lens, 2, 128, 128, 64, "bf16", "bf16")
    x = torch.randn(b.T, 4 + 4, 128, device="cuda").bfloat16()
    o = torch.full((b.T + 70, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T + 70, 4), 7.0, device="cuda")
    _, got, _ = check_attention(b, 4, q=x[:, :4], o=o[:b.T], lse=lse[:b.T])
    assert bool((o[b.T:] == 7).all()) and bool((lse[b.T:] == 7).all())
    dense, _ = jfa.jfa_paged_fwd(x[:, :4].contiguous(), *b.args())
    assert torch.equal(dense, got)


@pytest.mark.parametrize("new,lens", [([], []), ([0, 0], [5, 0]), ([3], [0]), ([4, 0, 2], [2, 9, 1])])
@pytest.mark.parametrize("cache", ["bf16", "mxfp8"])
def test_nothing_to_do(new, lens, cache):
    """No sequences, no new tokens, tokens that see no keys."""
    b = Batch(new, lens, 2, 64, 64, 16, cache, "bf16")
    check_attention(b, 4)
    check_attention(b, 4, causal=False)


def test_a_shared_page_and_the_same_page_twice():
    b = Batch([1, 1, 2], [100, 100, 90], 2, 128, 128, 32, "bf16", "bf16")
    b.table_h[1, :3] = b.table_h[0, :3]  # a common prefix
    b.table_h[2, 1] = b.table_h[2, 0]
    b.table.copy_(torch.tensor(b.table_h))
    check_attention(b, 8)


def _poisoned(b, hq):
    return (torch.full((b.T, hq, b.dv), 3.0, dtype=DT[b.dtype], device="cuda"),
            torch.full((b.T, hq), 3.0, device="cuda"))


@pytest.mark.parametrize("what", ["first", "order", "total", "negative", "long"])
@pytest.mark.parametrize("dtype,cache,new", [("f32", "f32", 2), ("bf16", "bf16", 1), ("bf16", "mxfp8", 60)])
def test_invalid_batches_compute_nothing(what, dtype, cache, new):
    b = Batch([new] * 5, [80] * 5, 2, 64, 64, 16, cache, dtype)
    if what == "first":
        b.offs[0] = 1
    elif what == "order":
        b.offs[2] = b.offs[4]
        b.offs[3] = b.offs[1]
    elif what == "total":
        b.offs[5] -= 1
    elif what == "negative":
        b.lens[3] = -1
    else:
        b.lens[1] = b.table.shape[1] * 16 + 1
    o, lse = _poisoned(b, 4)
    q = torch.randn(b.T, 4, 64, device="cuda").to(DT[dtype])
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, DT[dtype], heads_q=4))
    jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
    assert bool((o == 3).all()) and bool((lse == 3).all())
    # the planned calls on it compute nothing either
    before = b.cache.k.clone()
    jfa.jfa_cache_write(torch.ones(b.T, 2, 64, device="cuda", dtype=DT[dtype]),
                        torch.ones(b.T, 2, 64, device="cuda", dtype=DT[dtype]), *b.args(), ws=ws, planned=True)
    jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws, planned=True)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS
    assert bool((o == 3).all())
    assert torch.equal(before.view(torch.uint8), b.cache.k.view(torch.uint8))


@pytest.mark.parametrize("dtype,cache,new", [("f32", "f32", 1), ("bf16", "bf16", 1), ("bf16", "mxfp8", 1),
                                             ("bf16", "bf16", 60), ("bf16", "mxfp8", 60)])
def test_bad_pages_are_recorded_and_read_as_zeros(dtype, cache, new):
    b = Batch([new] * 4, [150] * 4, 2, 64, 64, 16, cache, dtype)
    bad = {1: 0, 3: 5}
    saved = b.k_h, b.v_h
    for s, j in bad.items():
        b.table_h[s, j] = b.pages if s == 1 else -1
    b.table.copy_(torch.tensor(b.table_h))
    # in the reference a bad page is a page of zeros
    b.k_h, b.v_h = (np.concatenate([x, np.zeros_like(x[:1])]) for x in saved)
    for s, j in bad.items():
        b.table_h[s, j] = b.pages
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, b.T, DT[dtype], heads_q=4))
    check_attention(b, 4, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES


def test_captured_steps_follow_their_inputs():
    """One captured step (norm-free: plan, attention) replayed with other lengths and tokens, on
    a stream of its own, while another stream uses a workspace of its own."""
    b = Batch([1] * 6, [300, 17, 64, 1, 129, 90], 2, 128, 128, 32, "bf16", "bf16")
    q = torch.randn(6, 8, 128, device="cuda").bfloat16()
    o, lse = _poisoned(b, 8)
    ws = jfa.paged_workspace(jfa.paged_params(b.cache, b.table, b.offs, b.lens, 6, torch.bfloat16, heads_q=8))
    jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jfa.jfa_paged_fwd(q, *b.args(), o=o, lse=lse, ws=ws)
    b2 = Batch([1] * 3, [200, 5, 77], 1, 64, 64, 16, "mxfp8", "bf16", seed=8)
    other = torch.cuda.Stream()
    for lens in ([300, 17, 64, 1, 129, 90], [10, 1, 64, 1, 100, 33], [299, 16, 2, 1, 128, 64]):
        b.lens_h[:] = lens
        b.lens.copy_(torch.tensor(lens))
        q.normal_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            check_attention(b2, 4)
        torch.cuda.synchronize()
        got, gl = o.clone(), lse.clone()
        _, want, wl = check_attention(b, 8, q=q)
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_cache_past_32_bits():
    """Pages whose elements lie past 2^32 (values and, in MXFP8, bytes)."""
    for kind, pages in (("bf16", 70000), ("mxfp8", 70000)):
        hk, page, d = 8, 64, 128
        if kind == "bf16":
            c = jfa.PagedCache(*(torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        else:
            u = lambda n: torch.empty(pages, hk, page, n, dtype=torch.uint8, device="cuda")
            c = jfa.PagedCache(u(d), u(d), u(d // 32), u(d // 32))
        assert c.k.numel() > 2 ** 32
        for new in (1, 200):
            n = [new, new]
            lens = [new + 150, new + 30]
            offs = torch.tensor([0, n[0], sum(n)], device="cuda")
            ln = torch.tensor(lens, device="cuda")
            W = max(-(-x // page) for x in lens)
            table = (pages - 1 - torch.arange(2 * W, device="cuda").int()).view(2, W).contiguous()
            rows = sum(lens)
            k, v = (torch.randn(rows, hk, d, device="cuda").bfloat16() for _ in range(2))
            full = torch.tensor([0, lens[0], rows], device="cuda")
            jfa.jfa_cache_write(k, v, c, table, full, ln)
            kr, vr = jfa.jfa_cache_read(c, table, full, ln, rows)
            if kind == "bf16":
                assert torch.equal(kr, k) and torch.equal(vr, v)
            q = torch.randn(sum(n), 16, d, device="cuda").bfloat16()
            o, lse = jfa.jfa_paged_fwd(q, c, table, offs, ln)
            kh, vh = f64(kr).transpose(1, 0, 2), f64(vr).transpose(1, 0, 2)
            at = [0, lens[0], rows]
            part = lambda x: (lambda b: x[:, at[b]:at[b + 1]])
            wo, wl, av, size = ref.paged(f64(q), part(kh), part(vh), [0, n[0], sum(n)], lens, 2, float(np.float32(d ** -0.5)), True)
            to, tl = ref.paged_bounds(wo, wl, av, size, d, max(lens), "bf16", True)
            assert np.all(np.abs(f64(o) - wo) <= to) and np.all(np.abs(f64(lse) - wl) <= tl)
        del c


# ------------------------------------------------------------------------------------ the cache
def rows_batch(new, lens, hk, dqk, dv, page, cache, dtype, seed=0):
    b = Batch(new, lens, hk, dqk, dv, page, cache, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    rn = lambda d: (torch.randn(b.T, hk, d, generator=g, device="cuda") * torch.exp(3 * torch.randn(b.T, hk, 1, generator=g, device="cuda"))).to(DT[dtype])
    return b, rn(dqk), rn(dv)


WRITES = [
    ("step", "bf16", "mxfp8", 8, 128, 128, 64),
    ("step", "bf16", "bf16", 2, 64, 128, 16),
    ("prompt", "bf16", "mxfp8", 3, 64, 32, 16),
    ("chunk", "f32", "mxfp8", 2, 128, 96, 128),
    ("chunk", "f32", "f32", 5, 24, 8, 32),
    ("chunk", "bf16", "bf16", 1, 256, 72, 256),
    ("prompt", "bf16", "mxfp8", 1, 256, 160, 32),
    ("many short", "bf16", "mxfp8", 4, 32, 32, 16),
]


@pytest.mark.parametrize("case", WRITES, ids=["%s-%s-%s-%d-D%d-%d-p%d" % c for c in WRITES])
def test_write_and_read_bit_for_bit(case):
    kind, dtype, cache, hk, dqk, dv, page = case
    b, k, v = rows_batch(*ragged(kind), hk, dqk, dv, page, cache, dtype)
    arrays = [a for a in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale) if a is not None]
    before = [a.view(torch.uint8).cpu().numpy().copy() for a in arrays]
    ws = jfa.jfa_cache_write(k, v, *b.args())
    assert jfa.jfa_status_check(ws) == jfa.JFA_OK
    after = [a.view(torch.uint8).cpu().numpy() for a in arrays]
    kr, vr = jfa.jfa_cache_read(*b.args(), b.T, dtype=DT[dtype])
    touched = np.zeros((b.pages, page), bool)
    want = [f64(k), f64(v)]
    seen = np.zeros(b.T, bool)
    for s in range(b.B):
        for i in range(int(b.new[s])):
            pos = int(b.lens_h[s] - b.new[s]) + i
            if pos >= 0:
                seen[b.offs_h[s] + i] = True
                touched[b.table_h[s, pos // page], pos % page] = True
    for a, z in zip(before, after):  # nothing else has changed
        keep = ~np.broadcast_to(touched[:, None, :, None], a.shape)
        assert np.array_equal(a[keep], z[keep])
    for n, (got, x) in enumerate(zip((kr, vr), want)):
        if cache == "mxfp8":
            x, _, e = ref.quantize_rows(x)
        x[~seen] = 0
        assert np.array_equal(f64(got), x)
    if cache == "mxfp8":  # codes and scales themselves
        for s in range(b.B):
            for i in range(int(b.new[s])):
                pos = int(b.lens_h[s] - b.new[s]) + i
                if pos < 0:
                    continue
                pg, r = b.table_h[s, pos // page], pos % page
                _, code, e = ref.quantize_rows(f64(k)[b.offs_h[s] + i])
                assert np.array_equal(ref._DECODE[after[0][pg, :, r]], code)
                assert np.array_equal(after[2][pg, :, r].astype(int) - 127, e)


def test_quantised_extremes():
    """Zeros, one huge value among small ones, the smallest and largest values, infinities and
    NaN: blocks keep to themselves."""
    b, k, v = rows_batch([8], [8], 1, 128, 32, 16, "mxfp8", "bf16")
    k.normal_()
    k[0] = 0
    k[1, 0, 3] = 3e38
    k[2, 0, 40] = -float("inf")
    k[3, 0, 70] = float("nan")
    k[4] = 1e-38
    k[5] = -3.3e38
    k[6, 0, :32] = torch.tensor([448.0, -448, 1, 2 ** -6, 2 ** -9, 2 ** -10, 1.0625, 1.1875] * 4)
    jfa.jfa_cache_write(k, v, *b.args())
    kr, _ = jfa.jfa_cache_read(*b.args(), 8, dtype=torch.float32)
    x, got = f64(k), f64(kr)
    fin = np.isfinite(x)
    want, _, _ = ref.quantize_rows(np.where(np.isfinite(x), x, 0.0))
    blocks = np.ones((8, 1, 4), bool)
    blocks[2, 0, 1] = blocks[3, 0, 2] = False  # the blocks with an infinity or a NaN
    same = np.repeat(blocks, 32, -1)
    assert np.array_equal(got[same], want[same])
    assert got[2, 0, 40] == -448 * 2.0 ** 119  # saturated
    assert np.isnan(got[3, 0, 70]) and np.isfinite(got[3, 0, 64:70]).all()
    # a NaN's block is scaled by its other values
    w, _, _ = ref.quantize_rows(np.where(fin, x, 0.0)[3])
    assert np.array_equal(got[3, 0, 71:96], w[0, 71:96])


def test_strided_rows_and_bad_pages_of_the_cache():
    b, k, v = rows_batch([4, 4], [20, 40], 2, 64, 64, 16, "bf16", "bf16")
    x = torch.randn(b.T, 2 + 2 + 2, 64, device="cuda").bfloat16()
    jfa.jfa_cache_write(x[:, 2:4], x[:, 4:], *b.args())
    kr, vr = jfa.jfa_cache_read(*b.args(), b.T)
    assert torch.equal(kr, x[:, 2:4]) and torch.equal(vr, x[:, 4:])
    b.table[1, 2] = b.pages + 5  # where sequence 1's new tokens go
    snap = b.cache.k.clone()
    ws = jfa.jfa_cache_write(k, v, *b.args())
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
    kr, vr = jfa.jfa_cache_read(*b.args(), b.T, ws=ws)
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_PAGES
    assert torch.equal(kr[:4], k[:4]) and bool((kr[4:] == 0).all()) and bool((vr[4:] == 0).all())
    changed = (snap.view(torch.int16) != b.cache.k.view(torch.int16)).flatten(1).any(1)
    assert set(torch.nonzero(changed).flatten().tolist()) <= {int(b.table_h[0, 1])}
    # invalid offsets: tokens outside every sequence are not written
    b.offs[1] = 100
    snap = b.cache.k.clone()
    ws = jfa.jfa_cache_write(k, v, *b.args())
    assert jfa.jfa_status_check(ws) == jfa.JFA_ERR_BAD_OFFSETS


# ------------------------------------------------------------------------------- the three together
@pytest.mark.parametrize("mxfp8", [False, True])
def test_prompt_then_steps(mxfp8):
    """Prompts and then single tokens of three sequences: norms and rotation, the cache, the
    attention, every step on one plan, against the whole computed in 64 bits from the rows that
    the cache holds."""
    hq, hk, D, page = 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    prompt, steps = [37, 1, 100], 3
    total = [n + steps for n in prompt]
    W = max(-(-n // page) for n in total)
    table = torch.randperm(3 * W, generator=g, device="cuda").int().view(3, W).contiguous()
    cache = jfa.paged_cache(3 * W, hk, D, page_size=page, mxfp8=mxfp8)
    wq, wk = 1 + 0.1 * rn(D), 1 + 0.1 * rn(D)
    rope = jfa.jfa_rope(D, layout="pairs")
    freq = ref.frequencies(D)
    done = np.zeros(3, np.int64)
    rows = [[[], []] for _ in range(3)]  # keys and values of every sequence, as the cache holds them
    for new in [prompt] + [[1, 1, 1]] * steps:
        offs_h = np.concatenate([[0], np.cumsum(new)])
        T = int(offs_h[-1])
        done = done + np.array(new)
        offs, lens = torch.tensor(offs_h, device="cuda"), torch.tensor(done, device="cuda")
        qkv = rn(T, hq + 2 * hk, D).bfloat16()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        pos_h = np.concatenate([np.arange(d - n, d) for d, n in zip(done, new)])
        yq, yk = jfa.jfa_norm_rope_fwd(q, k, torch.tensor(pos_h, device="cuda"), wq, wk, rope=rope)
        ws = jfa.jfa_paged_plan(yq, cache, table, offs, lens)
        jfa.jfa_cache_write(yk, v, cache, table, offs, lens, ws=ws, planned=True)
        o, lse = jfa.jfa_paged_fwd(yq, cache, table, offs, lens, ws=ws, planned=True)
        assert jfa.jfa_status_check(ws) == jfa.JFA_OK
        want, size = ref.norm_rope(f64(k), f64(wk), pos_h, freq, D, "pairs", 1.0, 1e-6)
        assert np.all(np.abs(f64(yk) - want) <= ref.HALF_STEP["bf16"] * np.abs(want) * 1.01 + 2e-6 * size)
        for x, n in ((f64(yk), 0), (f64(v), 1)):
            x = ref.quantize_rows(x)[0] if mxfp8 else x
            for b in range(3):
                rows[b][n].append(x[offs_h[b]:offs_h[b + 1]])
        of = lambda n: (lambda b: np.concatenate(rows[b][n]).transpose(1, 0, 2))
        wo, wl, av, size = ref.paged(f64(yq), of(0), of(1), offs_h, done, hq // hk, float(np.float32(D ** -0.5)), True)
        to, tl = ref.paged_bounds(wo, wl, av, size, D, int(done.max()), "bf16", True)
        assert np.all(np.abs(f64(o) - wo) <= to) and np.all(np.abs(f64(lse) - wl) <= tl)


def test_whole_prompts_match_the_dense_forward():
    """Whole prompts through the cache give what jfa_fwd gives on the same rows (each within its
    own bound: weights and result rounded to bf16)."""
    lens = [300, 17, 0, 513, 128]
    offs_h = np.concatenate([[0], np.cumsum(lens)])
    T, H, D, page = int(offs_h[-1]), 4, 128, 64
    q, k, v = (torch.randn(T, H, D, device="cuda").bfloat16() for _ in range(3))
    offs, ln = torch.tensor(offs_h, device="cuda"), torch.tensor(lens, device="cuda")
    W = max(-(-n // page) for n in lens)
    table = torch.arange(5 * W, device="cuda").int().view(5, W).contiguous()
    cache = jfa.paged_cache(5 * W, H, D, page_size=page)
    jfa.jfa_cache_write(k, v, cache, table, offs, ln)
    o, lse = jfa.jfa_paged_fwd(q, cache, table, offs, ln)
    wo, wl = jfa.jfa_fwd(q, k, v, offs, causal=True)
    assert float((lse - wl).abs().max()) <= 1e-4
    assert float((o.float() - wo.float()).abs().max()) <= 2 * 2.0 ** -8 * 5  # |o| and sum p |v| below 5 here
