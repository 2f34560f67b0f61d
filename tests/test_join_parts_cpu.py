"""The parts of tiles that the cuts of paged attention fall into, compiled for the host from the kernels' own source:
what the join looks up is what the CTAs' walks leave, also where a tile is cut into more parts than a warp has lanes."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from test_window_plan_cpu import CUDA, KERNELS, ROOT, tile, vp


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("host") / "parts.so")
    inc = [os.path.join(ROOT, "include"), os.path.join(ROOT, "jagged_attention_recsys_gb300", "csrc"), CUDA]
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-w", *("-I" + i for i in inc),
                    os.path.join(ROOT, "tests", "host", "join_parts_host.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.parts.restype = ctypes.c_int64
    return L


def parts(host, kernel, group, new, lens, window=0, sinks=0, heads_k=1, ctas=None):
    shape, most = tile(kernel, group)
    ctas = ctas or most
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    width = max(max(-(-n >> 6) for n in lens) + 1, 1)
    x = np.array([len(lens), offs[-1], width, 6, heads_k * group, heads_k, 1, window, sinks, *shape], np.int64)
    counts = np.zeros(ctas + 1, np.int64)
    wrong = host.parts(vp(x), vp(offs), vp(np.array(lens, np.int64)), ctas, ctas, vp(counts))
    return wrong, counts


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("n", [2, 3, 30, 31, 32, 33, 34, 63, 64, 65, 96, 97, 150])
def test_one_tile_in_so_many_parts(host, kernel, n):
    """One token over a long cache, cut for n CTAs: one tile, n parts."""
    wrong, counts = parts(host, kernel, 4, [1], [64 * 128 * n], ctas=n)
    assert wrong == 0 and counts[n] == 1 and counts.sum() == 1


@pytest.mark.parametrize("kernel", KERNELS)
def test_batches(host, kernel):
    rng = random.Random(8)
    seen = set()
    for _ in range(300):
        B = rng.choice([1, 2, 3, 8, 60])
        new = [rng.choice([0, 1, 2, 17, 300]) for _ in range(B)]
        lens = [max(0, m + rng.choice([0, -3, 40, 5000, 60000])) for m in new]
        window, sinks = rng.choice([(0, 0), (0, 0), (100, 4), (3000, 700)])
        wrong, counts = parts(host, kernel, rng.choice([1, 3, 4, 8]), new, lens, window, sinks, rng.choice([1, 2, 8]))
        assert wrong == 0
        seen |= set(np.nonzero(counts)[0].tolist())
    assert max(seen) > 64 and len(seen) > 20  # few parts and many
