"""The waits and arrivals of the paged attention's kernels, on the CPU, under random interleavings.

The stage ring of the paged attention's 16-row kernel (`csrc/paged_rows16.cu`), on the CPU: one
producer fills stages in order, each load lands at any later time, and the fills go in turn to
two pairs of consumers, which read and free them.  Every interleaving has to finish, and
every consumer has to find its own fill in the stage when its wait is over.

The 128-row kernel (`csrc/paged_tc.cu`): loader, the cleaner of the last block's values or MXFP8
converters, an MMA issuer and a softmax warpgroup for each stream, with loads that land in any
order and MMAs and commits that complete in their thread's order at any later time.  Every interleaving has to finish, and every role has to find in the shared
and tensor memory that it reads what its step needs."""
import random

import pytest

from test_barrier_protocols import Bar

WARPS = 4


def play(stages, segments, seed, own=lambda c, w, stages: c & 1 == w >> 1, limit=200000):
    """None, or what went wrong.  `segments`: blocks of each tile; the consumers meet at a tile's
    end.  `own`: whether fill c is warp w's, as one of two."""
    rng = random.Random(seed)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(2) for _ in range(stages)]
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
                if not own(f, w, stages):
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


@pytest.mark.parametrize("stages", [4, 6, 8, 16])
def test_every_consumer_reads_its_own_fill(stages):
    rng = random.Random(stages)
    for seed in range(60):
        segments = [rng.choice([0, 1, 2, 3, 5, 17, 40]) for _ in range(rng.randint(1, 8))]
        assert play(stages, segments, seed) is None


def test_stages_that_change_hands_are_caught():
    """With an odd number of stages a warp may meet another's fill that has not landed and take
    its parity for its own fill's."""
    assert any(play(5, [40], seed, limit=3000) for seed in range(40))


# ------------------------------------------------------------------------- the 128-row kernel
class Segment:
    """`blocks` key blocks; `split`: the streams share A's queries and take the blocks in turn,
    else A takes the first `n0` and B all."""

    def __init__(self, blocks, split, n0=0, tail=False):
        self.blocks, self.split, self.tail = blocks, split, tail
        self.n = [(blocks + 1) // 2, blocks // 2] if split else [min(n0, blocks), blocks]

    def block(self, x, i):
        return 2 * i + x if self.split else i


def play_tc(segments, stages, raws, seed, pass_all=True, pass_queries=True,
            limit=100000):
    """raws: stages of unconverted tiles (MXFP8), 0: tiles are loaded as they are used.
    pass_all=False: an issuer leaves out the stages that it does not use (and the user frees them
    twice).  pass_queries=False: B waits for A's queries without freeing them."""
    rng = random.Random(seed)
    B = lambda n, c=1: [Bar(c) for _ in range(n)]
    qfull, sfull, pfull, ofull, oempty = (B(2) for _ in range(5))
    qempty = [Bar(2 if pass_queries else 1), Bar(1)]
    xch_bar = Bar(1)
    full, empty, vtail, turn = B(stages), B(stages, 2), B(stages), B(2)
    rfull, rempty = B(max(raws, 1)), B(max(raws, 1))
    qmem, stage, raw = [None, None], [None] * stages, [None] * max(raws, 1)
    S, O = [None, None], [[], []]  # tensor memory: ("s" or "p", step) and the steps in O
    xch, flying, pipes = [None], [], [[], []]
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
                    tail = not raws and g.tail and kv and d == g.blocks - 1
                    fly(land((vtail if tail else f)[st], mem, st, (n, d, kv, "dirty") if tail else (n, d, kv)))
                    it += 1

    def cleaner():
        it, phase = 0, [0] * stages
        for n, g in segs:
            it += 2 * g.blocks
            if g.tail:
                st = (it - 1) % stages
                yield lambda: vtail[st].done(phase[st])
                phase[st] ^= 1
                need(stage[st] == (n, g.blocks - 1, 1, "dirty"), "cleans another tile")
                yield lambda: True
                stage[st] = (n, g.blocks - 1, 1)
                full[st].arrive()

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

    def issuer(x):
        it = p = o = qa = qb = tn = 0
        commit = lambda bar: pipes[x].append(bar.arrive)
        for n, g in segs:
            if g.n[0]:
                yield lambda: qfull[0].done(qa & 1)
                qa += 1
                if x and (not g.split or g.n[1] == 0) and pass_queries:
                    qempty[0].arrive()
            if x and not g.split:
                yield lambda: qfull[1].done(qb & 1)
                qb += 1
            qx, i = 0 if g.split else x, 0
            for d in range(g.blocks):
                mine = (d & 1) == x if g.split else d < g.n[x]
                for kv in (0, 1):
                    st, par = it % stages, (it // stages) & 1
                    it += 1
                    if not mine and not pass_all:
                        continue
                    passes = pass_all and (d == g.blocks - 1 if kv else d > 0)
                    if kv and pass_all:  # the streams take turns
                        yield lambda: turn[x].done((tn & 1) ^ (x == 0))
                        tn += 1
                    if mine and kv:
                        yield lambda: pfull[x].done(p & 1)
                        if i == 0:
                            yield lambda: oempty[x].done((o & 1) ^ 1)
                    yield lambda: full[st].done(par)
                    if passes:
                        pipes[x].append(turn[x ^ 1].arrive) if rng.random() < 0.5 else turn[x ^ 1].arrive()
                    if not mine:
                        empty[st].arrive()
                        continue
                    twice = not pass_all and (g.split or d >= g.n[0])
                    if kv == 0:
                        def run(i=i, st=st, d=d, n=n, qx=qx):
                            need(qmem[qx] == n and stage[st] == (n, d, 0), "S of other tiles")
                            need(S[x] is None or S[x][0] == "used", "S over weights in use")
                            S[x] = ("s", n, i)
                        pipes[x].append(run)
                        commit(sfull[x])
                        commit(empty[st])
                        if twice:
                            commit(empty[st])
                        if i == g.n[x] - 1:
                            if pass_queries or x == 0 or not g.split:
                                commit(qempty[qx])
                    else:
                        def run(i=i, st=st, d=d, n=n, qx=qx):
                            need(S[x] == ("p", n, i) and stage[st] == (n, d, 1), "P V of other tiles")
                            if i == 0:
                                need(O[x] in ([], ["read"]), "O over an output that was not read")
                                O[x] = []
                            O[x].append((n, d))
                            S[x] = ("used", n, i)
                        pipes[x].append(run)
                        if i == g.n[x] - 1:
                            commit(ofull[x])
                            o += 1
                        commit(empty[st])
                        if twice:
                            commit(empty[st])
                        p += 1
                        i += 1

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

    roles = {"loader": loader(), "issuer a": issuer(0), "issuer b": issuer(1), "a": softmax(0), "b": softmax(1)}
    roles["converter" if raws else "cleaner"] = converter() if raws else cleaner()
    waits = {k: (lambda: True) for k in roles}
    stuck = 0
    try:
        while roles:
            z = rng.random()
            if flying and z < 0.2:
                flying.pop(rng.randrange(len(flying)))()
                stuck = 0
            elif any(pipes) and z < 0.5:
                rng.choice([q for q in pipes if q]).pop(0)()
                stuck = 0
            k = rng.choice(sorted(roles))
            if not waits[k]():
                stuck += 1
                if stuck > limit and not flying and not any(pipes):
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
        out.append(Segment(blocks, split, max(0, blocks - rng.choice([0, 0, 1, 2, 20])), rng.random() < 0.4))
    return out


@pytest.mark.parametrize("stages,raws", [(5, 0), (8, 0), (3, 3), (6, 3)])
def test_streams_of_the_128_row_kernel(stages, raws):
    rng = random.Random(stages)
    for seed in range(150):
        assert play_tc(tc_segments(rng), stages, raws, seed) is None


def test_leaving_out_stages_is_caught():
    """An issuer that does not pass every stage takes older phases for its own."""
    segs = [Segment(24, True), Segment(24, True)]
    assert any(play_tc(segs, 6, 0, seed, pass_all=False, limit=3000) for seed in range(200))


def test_a_query_tile_that_one_issuer_does_not_free_is_caught():
    """B sees the phases of A's queries only if the loader waits for it."""
    rng = random.Random(2)
    assert any(play_tc(tc_segments(rng), 5, 0, seed, pass_queries=False, limit=3000) for seed in range(200))
