"""The paged attention's work plan under a window with sinks and over groups of sequences, compiled for
the host from the kernels' own source: every row meets each key that it sees exactly once, and the work
is cut evenly."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
KERNELS = ["rows8", "rows16", "tcgen05", "cores"]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("host") / "window.so")
    inc = [os.path.join(ROOT, "include"), os.path.join(ROOT, "jagged_attention_recsys_gb300", "csrc"), CUDA]
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-w", *("-I" + i for i in inc),
                    os.path.join(ROOT, "tests", "host", "window_plan_host.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.walk.restype = ctypes.c_int64
    return L


def tile(kernel, group):
    if kernel == "tcgen05":
        tokens = 2 * (128 // group)
        return [tokens * group, tokens, group, 1, 128, 192, 512], 152
    most = 8 if kernel == "rows8" and group <= 8 else 16
    gsub = min(group, most)
    tokens = most // gsub
    shape = [tokens * gsub, tokens, gsub, -(-group // gsub)]
    return (shape + [32, 32, 32], 456) if kernel == "cores" else (shape + [64, 64, 192], 304)


def vp(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def walk(host, kernel, group, new, lens, causal, window, sinks, page_shift, groups=None):
    shape, ctas = tile(kernel, group)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    T, width = int(offs[-1]), max(max(-(-n >> page_shift) for n in lens) + 1, 1)
    B = len(lens)
    x = np.array([B, T, width, page_shift, 2 * group, 2, causal, window, sinks, len(new), *shape], np.int64)
    top = max(max(lens), 1)
    met, written = np.zeros((T + 1, top), np.int32), np.zeros((T + 1, 2 * group), np.int64)
    busy = np.zeros(1, np.int64)
    lens, groups = np.array(lens, np.int64), None if groups is None else np.array(groups, np.int64)
    wrong = host.walk(vp(x), vp(offs), vp(lens), vp(groups), ctas, ctypes.c_int64(top), vp(met), vp(written), vp(busy))
    return wrong, met[:T], written[:T], int(busy[0]), ctas


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_visible_key_is_met_once(host, kernel):
    rng = random.Random(4)
    for _ in range(80):
        group, shift = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([4, 5, 6, 8])
        B, top = rng.choice([1, 2, 9]), rng.choice([1, 3, 200])
        new = [rng.randint(0, top) for _ in range(B)]
        lens = [max(0, n + rng.choice([0, 5, -3, 300, 900])) for n in new]
        window, sinks = rng.choice([1, 2, 63, 64, 65, 200, 5000, 2 ** 31 - 1]), rng.choice([0, 1, 4, 64, 130, 5000, 2 ** 31 - 1])
        wrong, met, written, _, _ = walk(host, kernel, group, new, lens, 1, window, sinks, shift)
        assert wrong == 0 and np.all(written == 1)
        t, k = 0, np.arange(met.shape[1])
        for n, m in zip(new, lens):
            for i in range(m - n, m):
                sees = (k <= i) & ((i - k < window) | (k < sinks))
                assert np.array_equal(met[t] > 0, sees) and met[t].max(initial=0) <= 1
                t += 1


def test_work_under_a_window_is_cut_evenly(host):
    """A CTA's share of a chunked batch: its blocks against the average's."""
    for kernel, new, lens in (("tcgen05", [1000] * 4, [1000, 3000, 1500, 4000]), ("rows16", [1] * 200, list(range(40, 4040, 20)))):
        wrong, met, _, busy, ctas = walk(host, kernel, 4, new, lens, 1, 600, 4, 6)
        shape, _ = tile(kernel, 4)
        # blocks that all CTAs walk: every tile's visible stretch, in blocks that it cuts
        total = 0
        for n, m in zip(new, lens):
            for first in range(m - n, m, shape[1]):
                low, end = max(0, first - 599), min(first + shape[1], m)
                total += -(-end // shape[4]) - low // shape[4] + (1 if low >= shape[4] else 0)
        total *= 2  # key heads
        assert wrong == 0 and busy <= 1.5 * total / ctas + 4


@pytest.mark.parametrize("kernel", KERNELS)
def test_groups_of_sequences(host, kernel):
    """Phase 1 of a shared prefix: a group's tokens are one sequence's, and see all of its keys."""
    rng = random.Random(5)
    for _ in range(60):
        group = rng.choice([1, 2, 4, 16])
        new = [rng.choice([0, 1, 1, 2, 40]) for _ in range(rng.choice([1, 5, 30]))]
        cuts = sorted(rng.randint(0, len(new)) for _ in range(rng.randint(0, 4)))
        groups = [0, *cuts, len(new)]
        prefix = [rng.choice([0, 1, 64, 500]) for _ in groups[1:]]
        wrong, met, written, _, _ = walk(host, kernel, group, new, prefix, 0, 0, 0, 6, groups)
        assert wrong == 0 and np.all(written == 1)
        t = 0
        for g, n in enumerate(prefix):
            for _ in range(sum(new[groups[g]:groups[g + 1]])):
                assert np.all(met[t, :n] == 1) and np.all(met[t, n:] == 0)
                t += 1
        for bad in (lambda x: x.__setitem__(0, 1), lambda x: x.__setitem__(-1, len(new) + 1), lambda x: x.__setitem__(-1, len(new) - 1),
                    lambda x: x.__setitem__(0, -1)):
            y = list(groups)
            bad(y)
            assert walk(host, kernel, group, new, prefix, 0, 0, 0, 6, y)[0] == -1
