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

CAPTURED = """
import numpy as np
import torch
from paged_kv_cache_395_b200 import pa
from tests import step_model
from tests.test_step_tables import BS, dev
B, M, N, T = 70, 40, 2500, 9000
rng = np.random.default_rng(3)
tables, lens = np.full((B, M), -1, np.int32), np.zeros(B, np.int32)
free, count = rng.permutation(N).astype(np.int32), N
t, l, f, c = dev(tables), dev(lens), dev(free), dev(np.array([count], np.int32))
n = torch.zeros(B, dtype=torch.int32, device="cuda")
slots, pos = torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
st = torch.cuda.Stream()
st.wait_stream(torch.cuda.current_stream())
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=st):     # the process's first call
    pa.pa_step_tables(t, l, n, f, c, slots, positions=pos)
for i in range(6):
    news = rng.integers(1, 100, B).astype(np.int32)
    news[rng.random(B) < 0.2] = -1
    news[rng.random(B) < 0.1] = 0
    n.copy_(dev(news))
    g.replay()
    tables, lens, free, count, _, s, p, _, flags = step_model.step(tables, lens, news, free, count, T)
    assert flags == 0 and pa.pa_get_error_flags(reset=True) == 0
    assert np.array_equal(slots.cpu().numpy(), s) and np.array_equal(pos.cpu().numpy(), p)
    assert np.array_equal(l.cpu().numpy(), lens) and int(c) == count and np.array_equal(f.cpu().numpy(), free)
    assert np.array_equal(t.cpu().numpy(), tables)
print("replayed")
"""


@pytest.mark.gpu
def test_a_step_of_many_tokens_captured_first():
    """Both launches captured by the first call of a process, and replayed."""
    r = subprocess.run([sys.executable, "-c", CAPTURED], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout == "replayed\n", r.stderr[-3000:]
