"""pa_step_tables around the batch sizes at which a kernel's shared memory passes the 48 KB that a
launch has without asking for more.  Each in a process of its own, smallest size first: a larger
call before would have asked already."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STEPS = """
import sys
import numpy as np
import torch
from tests.test_step_tables import BS, check
for B, T in {sizes}:
    rng = np.random.default_rng(B)
    M = 3
    lens = rng.integers(0, M * BS, B).astype(np.int32)
    news = rng.integers(-1, 2, B).astype(np.int32)
    nb = -(-lens // BS)
    N = int(nb.sum()) + B + 1
    perm = rng.permutation(N).astype(np.int32)
    tables = np.full((B, M), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    free = np.zeros(N, np.int32)
    free[:N - at] = perm[at:]
    check(tables, lens, news, free, N - at, T)
    print("served", B, T)
"""


def served(sizes):
    r = subprocess.run([sys.executable, "-c", STEPS.format(sizes=sizes)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    assert r.stdout.split("\n")[:-1] == [f"served {b} {t}" for b, t in sizes]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4096, 9000])
def test_batches_around_the_default_shared_memory(T):
    """The prefix sums take 25 bytes a sequence beside the kernel's own 400."""
    served([(b, T) for b in (1930, 1947, 1948, 1949, 1950, 1964, 1965)])


@pytest.mark.gpu
def test_slots_of_batches_around_the_default_shared_memory():
    """The launch that writes the slots of a step with many tokens takes 8 bytes a sequence beside
    its own 256."""
    served([(b, 9000) for b in (6111, 6112, 6113, 6144, 6145)])
