"""The paged attention's work plan, compiled for the host from the kernels' own source: every row is
computed over all the blocks it needs and written once, and calls on a plan of another request, or
on memory that holds none, meet no index outside their arrays."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("host") / "plan.so")
    inc = [os.path.join(ROOT, "include"), os.path.join(ROOT, "jagged_attention_recsys_gb300", "csrc"), CUDA]
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-w", *("-I" + i for i in inc),
                    os.path.join(ROOT, "tests", "host", "paged_plan_host.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.run.restype = ctypes.c_int64
    return L


class Request:
    """A batch with the tiles of one of the kernels."""

    def __init__(self, rng, kernel):
        self.hk = rng.choice([1, 2, 4])
        group = rng.choice([1, 2, 3, 4, 8, 16, 20])
        self.hq, B = self.hk * group, rng.choice([1, 2, 7, 40])
        self.page = 16
        top = rng.choice([1, 3, 300])
        self.new = [rng.randint(0, top) for _ in range(B)]
        self.lens = [max(0, n + rng.choice([0, 5, -3, 700, 4000])) for n in self.new]
        self.width = max(-(-n // self.page) for n in self.lens) + 1
        self.causal = rng.randint(0, 1)
        if kernel == "tcgen05":
            tokens = 2 * (128 // group)
            self.tile = [tokens * group, tokens, group, 1, 128, 192, 512]
            self.ctas = 152
        else:
            most = 8 if kernel == "rows8" and group <= 8 else 16
            gsub = min(group, most)
            tokens = most // gsub
            self.tile = [tokens * gsub, tokens, gsub, -(-group // gsub), 32, 64, 192]
            self.ctas = 456 if most == 8 else 304

    def arrays(self):
        offs = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)
        x = np.array([len(self.new), offs[-1], self.width, 4, self.hq, self.hk, self.causal, *self.tile], np.int64)
        return x, offs, np.array(self.lens, np.int64)


def vp(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def plan(host, r):
    x, offs, lens = r.arrays()
    pos, cum = np.zeros((r.ctas + 1, 4), np.int32), np.zeros(len(r.new) + 1, np.int64)
    assert host.plan(vp(x), vp(offs), vp(lens), r.ctas, vp(cum), vp(pos)) == 1
    return pos


def run(host, r, pos, offs=None, lens=None):
    x, o, n = r.arrays()
    offs, lens = (o if offs is None else offs), (n if lens is None else lens)
    blocks, written = (np.zeros(int(x[1]) * r.hq + 1, np.int64) for _ in range(2))
    bad = host.run(vp(x), vp(offs), vp(lens), r.ctas, vp(pos), vp(blocks), vp(written))
    return bad, blocks[:-1].reshape(-1, r.hq), written[:-1].reshape(-1, r.hq)


KERNELS = ["rows8", "rows16", "tcgen05"]


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_row_is_whole_and_written_once(host, kernel):
    rng = random.Random(1)
    for _ in range(60):
        r = Request(rng, kernel)
        bad, blocks, written = run(host, r, plan(host, r))
        assert bad == 0 and np.all(written == 1)
        t, keys = 0, r.tile[4]
        for n, m in zip(r.new, r.lens):
            for i in range(n):
                last = (i // r.tile[1] + 1) * r.tile[1]  # the tile's last token
                see = m if not r.causal else max(0, m - n + min(n, last))
                assert np.all(blocks[t + i] == -(-see // keys))
            t += n


def test_plans_of_other_requests_stay_inside_the_arrays(host):
    rng = random.Random(2)
    for _ in range(600):
        a, b = (Request(rng, rng.choice(KERNELS)) for _ in range(2))
        pos = plan(host, a)
        if len(pos) <= b.ctas:  # behind the plan: whatever was there
            rest = np.array([[rng.choice([0, 1, 7, -1, -2 ** 31, 2 ** 31 - 1]) for _ in range(4)]
                             for _ in range(b.ctas + 1 - len(pos))], np.int32)
            pos = np.concatenate([pos, rest])
        bad, _, _ = run(host, b, np.ascontiguousarray(pos))
        assert bad == 0


def test_changed_offsets_and_lengths_stay_inside_the_arrays(host):
    rng = random.Random(3)
    for _ in range(300):
        r = Request(rng, rng.choice(KERNELS))
        pos = plan(host, r)
        _, offs, lens = r.arrays()
        for a in (offs, lens):
            for _ in range(rng.randint(0, 2)):
                a[rng.randrange(len(a))] = rng.choice([-1, 0, 3, 10 ** 4, 2 ** 40, -2 ** 62, int(r.width) * r.page])
        bad, _, _ = run(host, r, pos, offs, lens)
        assert bad == 0
