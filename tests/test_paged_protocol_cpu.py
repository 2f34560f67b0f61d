"""The waits and arrivals of the paged attention's kernels, on the CPU, under random interleavings.

The stage ring of the paged attention's 16-row kernel (`csrc/paged_rows16.cu`), on the CPU: one
producer fills stages in order, each load lands at any later time, and the fills go in turn to
four consumers, each of which reads and frees its own.  Every interleaving has to finish, and
every consumer has to find its own fill in the stage when its wait is over.

The 128-row kernel (`csrc/paged_tc.cu`): loader, MXFP8 converters, MMA issuer and two softmax
warpgroups, with loads that land in any order and MMAs and commits that complete in issue order
at any later time.  Every interleaving has to finish, and every role has to find in the shared
and tensor memory that it reads what its step needs."""
import random

import pytest

from test_barrier_protocols import Bar

WARPS = 4


def play(stages, segments, seed, limit=200000):
    """None, or what went wrong.  `segments`: blocks of each tile; the consumers meet at a tile's
    end."""
    rng = random.Random(seed)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(1) for _ in range(stages)]
    holds = [None] * stages  # the fill that a stage holds
    flying = []              # loads on their way: (stage, fill)
    total = sum(segments)
    at_end = [0] * len(segments)
    gates = [sum(segments[:i + 1]) for i in range(len(segments))]

    def producer():
        for c in range(total):
            yield lambda: empty[c % stages].done(((c // stages) & 1) ^ 1)
            flying.append((c % stages, c))

    def consumer(w):
        c = 0
        for i, gate in enumerate(gates):
            for f in range(c, gate):
                if f % WARPS != w:
                    continue
                st, par = f % stages, (f // stages) & 1
                yield lambda: full[st].done(par)
                if holds[st] != f:
                    raise AssertionError("fill %d reads fill %s" % (f, holds[st]))
                yield lambda: True  # reading
                if holds[st] != f:
                    raise AssertionError("fill %d was overwritten" % f)
                empty[st].arrive()
            c = gate
            at_end[i] += 1
            yield lambda: at_end[i] == WARPS

    roles = {"producer": producer(), **{w: consumer(w) for w in range(WARPS)}}
    waits = {k: (lambda: True) for k in roles}
    stuck = 0
    try:
        while roles:
            if flying and rng.random() < 0.3:  # some load lands, not the oldest first
                st, c = flying.pop(rng.randrange(len(flying)))
                holds[st] = c
                full[st].arrive()
                stuck = 0
            k = rng.choice(sorted(roles, key=str))
            if not waits[k]():
                stuck += 1
                if stuck > limit and not flying:
                    return "stuck: %s" % sorted(roles, key=str)
                continue
            stuck = 0
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k], waits[k]
    except AssertionError as e:
        return str(e)
    return None


@pytest.mark.parametrize("stages", [4, 8, 12, 16])
def test_every_consumer_reads_its_own_fill(stages):
    rng = random.Random(stages)
    for seed in range(60):
        segments = [rng.choice([0, 1, 2, 3, 5, 17, 40]) for _ in range(rng.randint(1, 8))]
        assert play(stages, segments, seed) is None


def test_stages_that_change_hands_are_caught():
    """With a number of stages that the warps do not divide, a warp may meet another's fill that
    has not landed and take its parity for its own fill's."""
    assert any(play(5, [40], seed) for seed in range(40))


# ------------------------------------------------------------------------- the 128-row kernel
class Segment:
    """`blocks` key blocks; `split`: the streams share A's queries and take the blocks in turn,
    else A takes the first `n0` and B all."""

    def __init__(self, blocks, split, n0=0):
        self.blocks, self.split = blocks, split
        self.n = [(blocks + 1) // 2, blocks // 2] if split else [min(n0, blocks), blocks]

    def block(self, x, i):
        return 2 * i + x if self.split else i

    def both(self, d):
        return not self.split and d < self.n[0]


def play_tc(segments, stages, raws, seed, xch_early=False, limit=100000):
    """raws: stages of unconverted tiles (MXFP8), 0: tiles are loaded as they are used."""
    rng = random.Random(seed)
    B = lambda n, c=1: [Bar(c) for _ in range(n)]
    qfull, qempty, sfull, pfull, ofull, oempty = (B(2) for _ in range(6))
    xch_bar = Bar(1)
    full, empty = B(stages), B(stages, 2)
    rfull, rempty = B(max(raws, 1)), B(max(raws, 1))
    qmem, stage, raw = [None, None], [None] * stages, [None] * max(raws, 1)
    S, O = [None, None], [[], []]  # tensor memory: ("s" or "p", step) and the steps in O
    xch, flying, pipe, outputs = [None], [], [], []
    segs = [(n, g) for n, g in enumerate(segments) if g.blocks]

    def need(ok, what):
        if not ok:
            raise AssertionError(what)

    def fly(fn):
        flying.append(fn)

    def land(bar, mem, i, what):
        def fn():
            mem[i] = what
            bar.arrive()
        return fn

    def loader():
        it, q_it = 0, [0, 0]
        for n, g in segs:
            for x in (0, 1):
                if g.n[x] == 0 or (g.split and x):
                    continue
                yield lambda: qempty[x].done((q_it[x] & 1) ^ 1)
                fly(land(qfull[x], qmem, x, n))
                q_it[x] += 1
            for d in range(g.blocks):
                for kv in (0, 1):
                    f, e, mem, ring = (rfull, rempty, raw, raws) if raws else (full, empty, stage, stages)
                    st = it % ring
                    yield lambda: e[st].done(((it // ring) & 1) ^ 1)
                    fly(land(f[st], mem, st, (n, d, kv)))
                    it += 1

    def converter():
        it = 0
        for n, g in segs:
            for d in range(g.blocks):
                for kv in (0, 1):
                    rs, st = it % raws, it % stages
                    yield lambda: rfull[rs].done((it // raws) & 1)
                    yield lambda: empty[st].done(((it // stages) & 1) ^ 1)
                    need(raw[rs] == (n, d, kv), "converts another tile")
                    stage[st] = (n, d, kv)
                    full[st].arrive()
                    rempty[rs].arrive()
                    it += 1

    def issuer():
        base, q, p, o = 0, [0, 0], [0, 0], [0, 0]
        commit = lambda bar: pipe.append(bar.arrive)

        def scores(n, g, x, i):
            d, qx = g.block(x, i), 0 if g.split else x
            idx = base + 2 * d
            st = idx % stages
            if i == 0:
                yield lambda: qfull[qx].done(q[qx] & 1)
            yield lambda: full[st].done((idx // stages) & 1)

            def run():
                need(qmem[qx] == n and stage[st] == (n, d, 0), "S of other tiles")
                need(S[x] is None or S[x][0] == "used", "S over weights in use")
                S[x] = ("s", n, i)
            pipe.append(run)
            commit(sfull[x])
            commit(empty[st])
            if not g.both(d):
                commit(empty[st])
            if (d == g.blocks - 1) if g.split else (i == g.n[x] - 1):
                commit(qempty[qx])

        def output(n, g, x, i):
            d = g.block(x, i)
            idx = base + 2 * d + 1
            st = idx % stages
            yield lambda: pfull[x].done(p[x] & 1)
            yield lambda: full[st].done((idx // stages) & 1)
            if i == 0:
                yield lambda: oempty[x].done((o[x] & 1) ^ 1)
            p[x] += 1

            def run():
                need(S[x] == ("p", n, i) and stage[st] == (n, d, 1), "P V of other tiles")
                if i == 0:
                    need(O[x] in ([], ["read"]), "O over an output that was not read")
                    O[x] = []
                O[x].append((n, d))
                S[x] = ("used", n, i)
            pipe.append(run)
            commit(empty[st])
            if not g.both(d):
                commit(empty[st])
            if i == g.n[x] - 1:
                commit(ofull[x])
                o[x] += 1

        for n, g in segs:
            for x in (0, 1):
                if g.n[x]:
                    yield from scores(n, g, x, 0)
            for i in range(max(g.n)):
                for x in (0, 1):
                    if i < g.n[x]:
                        yield from output(n, g, x, i)
                        if i + 1 < g.n[x]:
                            yield from scores(n, g, x, i + 1)
            base += 2 * g.blocks
            q[0] += g.n[0] > 0
            q[1] += not g.split and g.n[1] > 0

    def softmax(x):
        s_it = o_it = x_it = 0
        for n, g in enumerate(segments):
            for i in range(g.n[x]):
                yield lambda: sfull[x].done(s_it & 1)
                need(S[x] == ("s", n, i), "reads other scores")
                need(i == 0 or len(O[x]) == i, "O moves while it may be rescaled")
                s_it += 1
                yield lambda: True
                S[x] = ("p", n, i)
                pfull[x].arrive()
            if g.split and x:
                if g.n[1]:
                    if xch_early:
                        xch[0] = n
                    yield lambda: ofull[1].done(o_it & 1)
                    o_it += 1
                    xch[0] = n
                    xch_bar.arrive()
                continue
            if g.n[x]:
                yield lambda: ofull[x].done(o_it & 1)
                o_it += 1
            if g.split and g.n[1]:
                yield lambda: xch_bar.done(x_it & 1)
                x_it += 1
                yield lambda: True
                need(xch[0] == n, "another tile's statistics")
            done = list(O[x]) if g.n[x] else []
            if g.split and g.n[1]:
                done += O[1]
            need(sorted(done) == [(n, g.block(x if not g.split else y, i)) for y in ((0, 1) if g.split else (x,))
                                  for i in range(g.n[y])] if not g.split else sorted(done) == [(n, d) for d in range(g.blocks)],
                 "an output of other steps")
            yield lambda: True
            if g.n[x]:
                O[x] = ["read"]
                oempty[x].arrive()
            if g.split and g.n[1]:
                O[1] = ["read"]
                oempty[1].arrive()

    roles = {"loader": loader(), "issuer": issuer(), "a": softmax(0), "b": softmax(1)}
    if raws:
        roles["converter"] = converter()
    waits = {k: (lambda: True) for k in roles}
    stuck = 0
    try:
        while roles:
            z = rng.random()
            if flying and z < 0.2:
                flying.pop(rng.randrange(len(flying)))()
                stuck = 0
            elif pipe and z < 0.5:
                pipe.pop(0)()
                stuck = 0
            k = rng.choice(sorted(roles))
            if not waits[k]():
                stuck += 1
                if stuck > limit and not flying and not pipe:
                    return "stuck: %s" % sorted(roles)
                continue
            stuck = 0
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k], waits[k]
    except AssertionError as e:
        return str(e)
    return None


def tc_segments(rng):
    out = []
    for _ in range(rng.randint(1, 7)):
        blocks = rng.choice([0, 1, 1, 2, 3, 6, 11])
        split = rng.random() < 0.5
        out.append(Segment(blocks, split, max(0, blocks - rng.choice([0, 0, 1, 2, 20]))))
    return out


@pytest.mark.parametrize("stages,raws", [(5, 0), (8, 0), (3, 3), (6, 3)])
def test_streams_of_the_128_row_kernel(stages, raws):
    rng = random.Random(stages)
    for seed in range(80):
        assert play_tc(tc_segments(rng), stages, raws, seed) is None


def test_an_early_handover_of_statistics_is_caught():
    """B writes its statistics before its product has waited for A: A may read the next tile's."""
    segs = [Segment(2, True)] * 6
    assert any(play_tc(segs, 5, 0, seed, xch_early=True) for seed in range(300))
