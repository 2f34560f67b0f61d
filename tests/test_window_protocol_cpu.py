"""Parts of the paged attention's 128-row kernel (`csrc/paged_tc.cuh`) on the CPU.  Over bf16 pages its loader
asks for a tile's queries behind the tile's first keys: the whole kernel's model with that order (over MXFP8
the queries go first, as in the model itself).  And under a window:

The ring of the paged attention's 128-row kernel under a window (`csrc/paged_tc.cuh`), on the CPU: tiles of
values of which some keys are hidden from every row, the sinks' block and the window's first among them,
land on a barrier of their own and become full once a cleaner has zeroed those rows.  Every random interleaving
of the loader, the loads, the cleaner and the two readers has to finish, and no reader may find a tile that is
another's or not clean."""
import inspect
import random

import pytest

import test_paged_protocol_cpu as model
from test_barrier_protocols import Bar


def play(segments, stages, seed, clean_all=True, limit=20000):
    """segments: of each, whether the values of its blocks have hidden keys.  clean_all=False: the cleaner looks
    at the last block alone, as without a window."""
    rng = random.Random(seed)
    full, empty, tail = [Bar(1) for _ in range(stages)], [Bar(2) for _ in range(stages)], [Bar(1) for _ in range(stages)]
    holds, flying = [None] * stages, []

    def land(bar, st, what):
        def fn():
            holds[st] = what
            bar.arrive()
        return fn

    def loader():
        it = 0
        for n, dirty in enumerate(segments):
            for d, hidden in enumerate(dirty):
                for kv in (0, 1):
                    st = it % stages
                    yield lambda: empty[st].done(((it // stages) & 1) ^ 1)
                    lands = tail if kv and hidden else full
                    flying.append(land(lands[st], st, (n, d, kv, "dirty" if kv and hidden else "")))
                    it += 1

    def cleaner():
        it, phase = 0, 0
        for n, dirty in enumerate(segments):
            for d in range(len(dirty)) if clean_all else range(max(0, len(dirty) - 1), len(dirty)):
                if not dirty[d]:
                    continue
                st = (it + 2 * d + 1) % stages
                yield lambda: tail[st].done((phase >> st) & 1)
                phase ^= 1 << st
                if holds[st] != (n, d, 1, "dirty"):
                    raise AssertionError("cleans another tile")
                yield lambda: True
                holds[st] = (n, d, 1, "")
                full[st].arrive()
            it += 2 * len(dirty)

    def reader():
        it = 0
        for n, dirty in enumerate(segments):
            for d in range(len(dirty)):
                for kv in (0, 1):
                    st = it % stages
                    yield lambda: full[st].done((it // stages) & 1)
                    if holds[st] != (n, d, kv, ""):
                        raise AssertionError("reads another tile")
                    yield lambda: True
                    empty[st].arrive()
                    it += 1

    roles = {"loader": loader(), "cleaner": cleaner(), "a": reader(), "b": reader()}
    waits = {k: (lambda: True) for k in roles}
    stuck = 0
    try:
        while roles:
            if flying and rng.random() < 0.3:
                flying.pop(rng.randrange(len(flying)))()
                stuck = 0
            k = rng.choice(sorted(roles))
            if not waits[k]():
                stuck += 1
                if stuck > limit and not flying:
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


def segments(rng):
    out = []
    for _ in range(rng.randint(1, 8)):
        n = rng.choice([0, 1, 2, 3, 7, 18])
        # the sinks' block, the window's first one or two, the last one
        out.append([rng.random() < (0.7 if i in (0, 1, 2, n - 1) else 0.02) for i in range(n)])
    return out


@pytest.mark.parametrize("stages", [3, 5, 8])
def test_cleaned_tiles(stages):
    rng = random.Random(stages)
    for seed in range(200):
        assert play(segments(rng), stages, seed) is None


def test_a_cleaner_of_the_last_block_alone_is_caught():
    rng = random.Random(1)
    assert any(play(segments(rng), 5, seed, clean_all=False, limit=3000) for seed in range(20))


QUERIES = '''            for x in (0, 1):
                if g.n[x] == 0 or (g.split and x):
                    continue
                yield lambda: qempty[x].done((q_it[x] & 1) ^ 1)
                fly(land(qfull[x], qmem, x, n))
                q_it[x] += 1
'''
RING = '''                for kv in (0, 1):
                    f, e, mem, ring = (rfull, rempty, raw, raws) if raws else (full, empty, stage, stages)
'''


def with_keys_first():
    """The model of the kernel with the loader's order over bf16 pages."""
    source = inspect.getsource(model.play_tc)
    assert source.count(QUERIES) == 1 and source.count(RING) == 1
    late = " " * 20 + "if d == 0 and kv == 1:\n" + "".join(" " * 12 + line + "\n" for line in QUERIES.splitlines())
    source = source.replace(QUERIES, "")
    head, body = RING.split("\n", 1)
    source = source.replace(RING, head + "\n" + late + body)
    space = dict(vars(model))
    exec(compile(source, "model", "exec"), space)
    return space["play_tc"]


@pytest.mark.parametrize("stages,raws", [(5, 0), (8, 0)])
def test_queries_behind_the_first_keys(stages, raws):
    play_tc = with_keys_first()
    rng = random.Random(stages + 100)
    for seed in range(150):
        assert play_tc(model.tc_segments(rng), stages, raws, seed) is None
