"""pa_step_tables: the plain model against the host's BlockManager, refusals (CPU), and
the kernel against the model, bit for bit (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_395_b200 import pa
from paged_kv_cache_395_b200.block_manager import BlockManager

from . import step_model

BS = 16


def trace(B, M, N, steps, seed, finish=0.1, prompt=60, share=False):
    """A decode loop on the host's manager: yields the step's inputs and what the manager
    did (tables of the live rows, slots, lengths, free list, refcounts)."""
    rng = np.random.default_rng(seed)
    bm = BlockManager(N, free_order=rng.permutation(N))
    ids, nxt = [None] * B, 0
    tables = np.full((B, M), -1, np.int32)
    if share:  # sequences 0 and 1 share full blocks with a prefix that the manager holds
        bm.add_sequence("prefix", 2 * BS)
        for b in (0, 1):
            bm.fork("prefix", b)
            ids[b], nxt = b, 2
            tables[b, :2] = bm.tables[b]
    for _ in range(steps):
        lens = np.array([bm.lens[s] if s is not None else 0 for s in ids], np.int32)
        news = np.zeros(B, np.int32)
        for b in range(B):
            if ids[b] is None:
                news[b] = rng.integers(0, min(prompt, M * BS) + 1)
            elif rng.random() < finish or lens[b] + 1 > M * BS:
                news[b] = -1
            else:
                news[b] = 1
        free, refs = np.array(bm._free + bm._deferred, np.int32), bm.refcount.astype(np.int32)
        before = (tables.copy(), lens, news, free, refs)
        for b in range(B):
            if news[b] == -1:
                bm.free_sequence(ids[b])
                ids[b] = None
        slots = []
        for b in range(B):
            if news[b] > 0 and ids[b] is None:
                slots += bm.add_sequence(nxt, int(news[b])).tolist()
                ids[b], nxt = nxt, nxt + 1
            elif news[b] > 0:
                slot, cow = bm.append_slot(ids[b])
                assert cow is None
                slots.append(slot)
            if ids[b] is not None:
                tables[b, :len(bm.tables[ids[b]])] = bm.tables[ids[b]]
        yield before, tables.copy(), slots, [bm.lens[s] if s is not None else 0 for s in ids], \
            list(bm._free), bm.refcount.copy()


@pytest.mark.parametrize("seed,share", [(0, False), (1, True), (2, True)])
def test_model_is_the_block_manager(seed, share):
    for before, tables, slots, lens, free, refs in trace(7, 6, 80, 40, seed, share=share):
        t0, l0, n0, f0, r0 = before
        full = np.zeros(80, np.int32)
        full[:len(f0)] = f0
        t, l, f, c, r, s, p, starts, flags = step_model.step(t0, l0, n0, full, len(f0), 512, r0)
        assert flags == 0 and l.tolist() == lens and s[:len(slots)].tolist() == slots and (s[len(slots):] == -1).all()
        assert f[:c].tolist() == free and r.tolist() == refs.tolist()
        assert starts[-1] == len(slots)
        for b, n in enumerate(lens):
            k = -(-n // BS)
            assert t[b, :k].tolist() == tables[b, :k].tolist()


# ---------------------------------------------------------------------------
# refusals (no GPU)
# ---------------------------------------------------------------------------
FAKE = 0x1000


def call(**kw):
    a = dict(tables=FAKE, lens=FAKE, news=FAKE, lens_out=FAKE, free=FAKE, count=FAKE, count_out=FAKE, refs=None,
             slots=FAKE, pos=None, starts=None, B=4, M=8, N=64, T=16, bs=16)
    a.update(kw)
    return pa.lib.pa_step_tables(*[ctypes.c_void_p(v) if k not in ("B", "M", "N", "T", "bs") else v
                                   for k, v in a.items()], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), pa.PA_ERR_SHAPE), (dict(M=0), pa.PA_ERR_SHAPE), (dict(N=0), pa.PA_ERR_SHAPE),
    (dict(T=-1), pa.PA_ERR_SHAPE), (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(B=pa.PA_STEP_MAX_SEQS + 1), pa.PA_ERR_UNSUPPORTED), (dict(B=64, M=1 << 25), pa.PA_ERR_UNSUPPORTED),
    (dict(N=1 << 31), pa.PA_ERR_UNSUPPORTED), (dict(T=(1 << 31) - 1), pa.PA_ERR_UNSUPPORTED),
    (dict(tables=None), pa.PA_ERR_NULL), (dict(lens=None), pa.PA_ERR_NULL), (dict(news=None), pa.PA_ERR_NULL),
    (dict(lens_out=None), pa.PA_ERR_NULL), (dict(free=None), pa.PA_ERR_NULL), (dict(count=None), pa.PA_ERR_NULL),
    (dict(count_out=None), pa.PA_ERR_NULL), (dict(slots=None), pa.PA_ERR_NULL),
])
def test_refusals(kw, status):
    assert call(**kw) == status


def test_python_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_step_tables(z.view(2, 2), z[:2], z[:2], z, z[:1], z.long())


# ---------------------------------------------------------------------------
# the kernel
# ---------------------------------------------------------------------------
def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_kernel(tables, lens, news, free, count, T, refs=None, in_place=False):
    t, l, n, f, c = dev(tables), dev(lens), dev(news), dev(free), dev(np.array([count], np.int32))
    r = None if refs is None else dev(refs)
    slots = torch.full((T,), 7, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    starts = torch.full((len(lens) + 1,), 7, dtype=torch.int32, device="cuda")
    lo = l if in_place else torch.full_like(l, 7)
    co = c if in_place else torch.full_like(c, 7)
    pa.pa_get_error_flags(reset=True)
    pa.pa_step_tables(t, l, n, f, c, slots, None if in_place else lo, None if in_place else co, pos, starts, r)
    flags = pa.pa_get_error_flags(reset=True)
    return [x if x is None else x.cpu().numpy() for x in (t, lo, f, co, r, slots, pos, starts)] + [flags]


def check(tables, lens, news, free, count, T, refs=None, **kw):
    want = step_model.step(tables, lens, news, free, count, T, refs)
    got = run_kernel(tables, lens, news, free, count, T, refs, **kw)
    names = ("tables", "lens", "free", "count", "refs", "slots", "positions", "row_starts", "flags")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(np.ravel(g), np.ravel(w)) if w is not None else g is None, name
    return want


def random_step(rng, B, M, prompt, refs, spare=1.0, bad=False):
    """A step of B rows: some finished, some new, some one token, some idle."""
    lens = rng.integers(0, M * BS + 1, B).astype(np.int32)
    news = np.ones(B, np.int32)
    kind = rng.random(B)
    news[kind < 0.2] = -1
    idle = (kind >= 0.2) & (kind < 0.3)
    news[idle] = 0
    fresh = (kind >= 0.3) & (kind < 0.5)
    lens[fresh] = 0
    news[fresh] = rng.integers(1, max(2, min(prompt, M * BS) + 1), int(fresh.sum()))
    if not bad:
        news = np.where((news > 0) & (lens + news > M * BS), -1, news).astype(np.int32)
    nb = -(-lens // BS)
    used = int(nb.sum())
    N = used + int(spare * (B * 4 + int(np.maximum(news, 0).sum()) // BS)) + 1
    perm = rng.permutation(N).astype(np.int32)
    tables = rng.integers(-5, 2 * N, (B, M)).astype(np.int32)  # beyond the rows: never read
    at = 0
    for b in range(B):
        tables[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    free = rng.integers(0, N, N).astype(np.int32)
    free[:N - used] = perm[used:]
    r = None
    if refs:
        r = np.zeros(N, np.int32)
        r[perm[:used]] = 1
        more = rng.random(N) < 0.1
        r[perm[:used][more[:used]]] += 1
        for b in range(B):  # some rows share their first blocks with the row before
            if b and min(nb[b], nb[b - 1]) > 1 and rng.random() < 0.3:
                for j in range(int(min(nb[b], nb[b - 1])) - 1):
                    r[tables[b, j]] -= 1
                    tables[b, j] = tables[b - 1, j]
                    r[tables[b, j]] += 1
        r = np.maximum(r, 0)
        for b in range(B):
            if lens[b] % BS and rng.random() < 0.9:
                r[tables[b, nb[b] - 1]] = 1
    return tables, lens, news, free, N - used, r


@pytest.mark.gpu
@pytest.mark.parametrize("refs", [False, True])
@pytest.mark.parametrize("B,M,prompt,slack", [(1, 1, 16, 0), (1, 300, 4800, 5), (3, 2, 9, 1), (64, 264, 40, 64),
                                              (255, 7, 100, 0), (257, 33, 500, 3), (1024, 12, 190, 1000),
                                              (8192, 5, 30, 7)])
def test_random_steps(B, M, prompt, slack, refs):
    rng = np.random.default_rng(B * 7 + refs)
    for i in range(3):
        t, l, n, f, c, r = random_step(rng, B, M, prompt, refs)
        check(t, l, n, f, c, int(np.maximum(n, 0).sum()) + slack, r, in_place=bool(i & 1))


@pytest.mark.gpu
@pytest.mark.parametrize("refs", [False, True])
def test_the_list_runs_out(refs):
    rng = np.random.default_rng(5)
    hit = 0
    for i in range(6):
        t, l, n, f, c, r = random_step(rng, 90, 20, 300, refs, spare=0.1 * i)
        w = check(t, l, n, f, c, int(np.maximum(n, 0).sum()) + 3, r)
        hit += bool(w[-1] & pa.PA_EFLAG_OUT_OF_BLOCKS)
    assert hit


@pytest.mark.gpu
def test_bad_rows_are_left_alone():
    t = np.arange(24, dtype=np.int32).reshape(6, 4)
    free = np.zeros(64, np.int32)
    free[:30] = np.arange(30, 60)
    cases = [
        ([-3, 5, 70, 20, 64, 0], [1, -2, 1, 50, 1, 2147483647]),    # lengths out of range, sums past the row
        ([5, 5, 5, 5, 5, 5], [1, 1, 1, 1, 1, 20]),                  # tokens past the slot buffer
        ([0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0]),
        ([64, 64, 64, 1, 1, 1], [-1, -1, -1, -1, -1, -1]),
    ]
    for lens, news in cases:
        check(t, np.array(lens, np.int32), np.array(news, np.int32), free, 30, 10)
    bad = t.copy()
    bad[0, 0], bad[1, 1], bad[2, 0] = -1, 64, 1 << 30
    w = check(bad, np.array([5, 20, 40, 3, 0, 16], np.int32), np.array([1, 1, -1, 1, 3, 1], np.int32), free, 30, 20)
    assert w[-1] & pa.PA_EFLAG_BAD_BLOCK
    for count in (-1, 65, 64, 0):
        check(t, np.array([5, 16, 0, 0, 0, 0], np.int32), np.array([-1, 1, 3, 0, 0, 0], np.int32), free, count, 8)


@pytest.mark.gpu
def test_counts_of_shared_blocks():
    # rows 0, 1 and 2 share block 0; row 2 holds block 1 twice; block 9 was free already
    t = np.array([[0, 2, -1], [0, 3, -1], [0, 1, 1], [9, -1, -1], [4, -1, -1]], np.int32)
    refs = np.zeros(16, np.int32)
    refs[[0, 1, 2, 3, 4]] = [3, 2, 1, 1, 2]
    free = np.zeros(16, np.int32)
    free[:3] = [9, 10, 11]
    lens = np.array([32, 32, 48, 16, 5], np.int32)
    for news in ([-1, 1, -1, 0, 1], [-1, -1, -1, 0, -1], [-1, -1, -1, -1, 0], [0, 0, -1, 0, 1]):
        check(t, lens, np.array(news, np.int32), free, 3, 4, refs)


@pytest.mark.gpu
@pytest.mark.parametrize("refs", [False, True])
def test_rows_that_are_not_served_in_a_step_of_many_tokens(refs):
    """The slots of a long token buffer are written by a launch of their own."""
    rng = np.random.default_rng(6)
    hit = 0
    for i in range(6):
        t, l, n, f, c, r = random_step(rng, 200, 40, 600, refs, spare=0.15 * i, bad=True)
        total = int(np.maximum(n, 0).sum())
        w = check(t, l, n, f, c, max(4097, total - 300 * (i & 1)), r, in_place=bool(i & 2))
        hit |= w[-1]
    assert hit & pa.PA_EFLAG_OUT_OF_BLOCKS and hit & pa.PA_EFLAG_BAD_LENGTH


@pytest.mark.gpu
def test_entries_outside_the_pool_on_the_list():
    for T in (40, 5000):
        t, free = np.full((3, 4), -1, np.int32), np.array([5, 9, -1, 4, 8, 2], np.int32)
        got = run_kernel(t, np.array([0, 16, 0], np.int32), np.array([20, 1, 16], np.int32), free, 5, T)
        assert got[-1] == pa.PA_EFLAG_BAD_BLOCK
        assert got[0][0, 1] == 4 and got[0][1, 1] == -1 and got[0][2, 0] == 9 and got[3][0] == 1
        assert (got[5] < 6 * BS).all() and (got[5][:16] == -1).all() and got[5][20] == -1
        assert got[1].tolist() == [20, 17, 16]


@pytest.mark.gpu
def test_empty_batch_and_no_slots():
    e = np.zeros((0, 3), np.int32)
    z = np.zeros(0, np.int32)
    got = run_kernel(e, z, z, np.arange(8, dtype=np.int32), 5, 6)
    assert got[3][0] == 5 and (got[5] == -1).all() and (got[6] == -1).all() and got[7].tolist() == [0]
    got = run_kernel(e, z, z, np.arange(8, dtype=np.int32), 5, 9000)
    assert got[3][0] == 5 and (got[5] == -1).all() and (got[6] == -1).all() and got[7].tolist() == [0]
    check(np.array([[3, 4]], np.int32), np.array([20], np.int32), np.array([-1], np.int32),
          np.array([0, 1, 2, 0, 0], np.int32), 3, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("share", [False, True])
def test_a_loop_of_steps_follows_the_block_manager(share):
    """The state stays on the device; every step's result is the host manager's."""
    B, M, N, T = 9, 6, 90, 600
    t = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    state = None
    pa.pa_get_error_flags(reset=True)
    for before, tables, slots, lens, free, refs in trace(B, M, N, 30, 11, share=share):
        t0, l0, n0, f0, r0 = before
        if state is None:
            f = np.zeros(N, np.int32)
            f[:len(f0)] = f0
            t.copy_(dev(t0))
            state = [dev(l0), dev(f), dev(np.array([len(f0)], np.int32)), dev(r0)]
        l, f, c, r = state
        s = torch.empty(T, dtype=torch.int64, device="cuda")
        pa.pa_step_tables(t, l, dev(n0), f, c, s, refcounts=r)
        assert s.cpu().numpy()[:len(slots)].tolist() == slots and l.cpu().tolist() == lens
        assert f.cpu().numpy()[:int(c)].tolist() == free and r.cpu().tolist() == refs.tolist()
        for b, n in enumerate(lens):
            assert t[b, :-(-n // BS)].cpu().tolist() == tables[b, :-(-n // BS)].tolist()
    assert pa.pa_get_error_flags(reset=True) == 0


@pytest.mark.gpu
def test_captured_steps():
    """One captured decode step, replayed: lengths grow and blocks come off the list in place."""
    B, M, N = 5, 4, 40
    lens = torch.tensor([0, 15, 16, 3, 31], dtype=torch.int32, device="cuda")
    news = torch.ones(B, dtype=torch.int32, device="cuda")
    t = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    t[1, 0], t[2, 0], t[3, 0], t[4, 0], t[4, 1] = 0, 1, 2, 3, 4
    free = torch.arange(5, 45, dtype=torch.int32, device="cuda")[:N] % N
    count = torch.tensor([N - 5], dtype=torch.int32, device="cuda")
    slots = torch.empty(8, dtype=torch.int64, device="cuda")
    model = [x.cpu().numpy() for x in (t, lens, free)] + [N - 5]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            pa.pa_step_tables(t, lens, news, free, count, slots)
    for _ in range(20):
        g.replay()
        mt, ml, mf, mc, _, ms, _, _, _ = step_model.step(model[0], model[1], np.ones(B, np.int32), model[2], model[3], 8)
        model = [mt, ml, mf, mc]
        torch.cuda.synchronize()
        assert slots.cpu().numpy().tolist() == ms.tolist() and lens.cpu().tolist() == ml.tolist()
        assert int(count) == mc and np.array_equal(t.cpu().numpy(), mt)
