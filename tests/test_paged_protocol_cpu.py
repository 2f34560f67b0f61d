"""The stage ring of the paged attention's 16-row kernel (`csrc/paged_rows16.cu`), on the CPU: one
producer fills stages in order, each load lands at any later time, and the fills go in turn to
four consumers, each of which reads and frees its own.  Every interleaving has to finish, and
every consumer has to find its own fill in the stage when its wait is over."""
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
