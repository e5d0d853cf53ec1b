"""pa_block_bounds and pa_select_blocks: refusals (CPU); boxes and choices against the
numpy model, bit for bit (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_395_b200 import pa

from . import sparse_model as M

BS = 16
FAKE = 0x1000
TD = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16, "int8": torch.int8}


def sparse_params(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=4,
                num_blocks=8, max_seq_len=64, q_dtype=pa.PA_F16, kv_dtype=pa.PA_F16, query_len=1, max_selected=4,
                sink_blocks=1, recent_blocks=1, flags=0)
    base.update(kw)
    p = pa.PaSparseParams()
    for k, v in base.items():
        setattr(p, k, v)
    return p


BAD_SPARSE = [
    (dict(num_seqs=-1), pa.PA_ERR_SHAPE), (dict(num_q_heads=6, num_kv_heads=4), pa.PA_ERR_SHAPE),
    (dict(num_kv_heads=0), pa.PA_ERR_SHAPE), (dict(query_len=-1), pa.PA_ERR_SHAPE), (dict(max_seq_len=-1), pa.PA_ERR_SHAPE),
    (dict(max_selected=0), pa.PA_ERR_SHAPE), (dict(recent_blocks=0), pa.PA_ERR_SHAPE),
    (dict(sink_blocks=-1), pa.PA_ERR_SHAPE), (dict(sink_blocks=3, recent_blocks=2), pa.PA_ERR_SHAPE),
    (dict(sink_blocks=2147483647, recent_blocks=2147483647), pa.PA_ERR_SHAPE),
    (dict(q_dtype=pa.PA_I8), pa.PA_ERR_DTYPE), (dict(q_dtype=pa.PA_F32), pa.PA_ERR_DTYPE),
    (dict(kv_dtype=pa.PA_I4), pa.PA_ERR_DTYPE), (dict(kv_dtype=pa.PA_BF16), pa.PA_ERR_DTYPE),
    (dict(head_dim=96), pa.PA_ERR_UNSUPPORTED), (dict(block_size=32), pa.PA_ERR_UNSUPPORTED),
    (dict(num_q_heads=130), pa.PA_ERR_UNSUPPORTED), (dict(flags=1), pa.PA_ERR_UNSUPPORTED),
    (dict(max_seq_len=pa.PA_SPARSE_MAX_SEQ_LEN + 1, max_blocks_per_seq=40000), pa.PA_ERR_UNSUPPORTED),
    (dict(max_selected=40000), pa.PA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_SPARSE)
def test_select_refusals(kw, status):
    p = sparse_params(**kw)
    assert pa.lib.pa_select_blocks(*[ctypes.c_void_p(FAKE)] * 7, ctypes.byref(p), None) == status


def test_select_pointers():
    p = sparse_params()
    assert pa.lib.pa_select_blocks(*[ctypes.c_void_p(FAKE)] * 7, None, None) == pa.PA_ERR_NULL
    for i in range(7):
        args = [ctypes.c_void_p(None if k == i else FAKE) for k in range(7)]
        assert pa.lib.pa_select_blocks(*args, ctypes.byref(p), None) == pa.PA_ERR_NULL
    args = [ctypes.c_void_p(FAKE + 8 * (k == 3)) for k in range(7)]
    assert pa.lib.pa_select_blocks(*args, ctypes.byref(p), None) == pa.PA_ERR_ALIGN
    assert pa.lib.pa_select_blocks(*[None] * 7, ctypes.byref(sparse_params(num_seqs=0)), None) == pa.PA_OK


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), pa.PA_ERR_SHAPE), (dict(H=0), pa.PA_ERR_SHAPE), (dict(N=0), pa.PA_ERR_SHAPE), (dict(M=0), pa.PA_ERR_SHAPE),
    (dict(new=-1), pa.PA_ERR_SHAPE), (dict(dt=pa.PA_I4), pa.PA_ERR_DTYPE), (dict(dt=9), pa.PA_ERR_DTYPE),
    (dict(d=80), pa.PA_ERR_UNSUPPORTED), (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(dt=pa.PA_I8, ks=None), pa.PA_ERR_NULL), (dict(bounds=None), pa.PA_ERR_NULL), (dict(scales=None), pa.PA_ERR_NULL),
    (dict(kc=None), pa.PA_ERR_NULL), (dict(tables=None), pa.PA_ERR_NULL), (dict(lens=None), pa.PA_ERR_NULL),
    (dict(kc=FAKE + 2), pa.PA_ERR_ALIGN), (dict(bounds=FAKE + 8), pa.PA_ERR_ALIGN),
    (dict(B=0, kc=None), pa.PA_OK), (dict(new=0, kc=None), pa.PA_OK),
])
def test_bounds_refusals(kw, status):
    a = dict(bounds=FAKE, scales=FAKE, kc=FAKE, ks=FAKE, tables=FAKE, first=None, lens=FAKE, B=2, H=2, d=64, bs=16, M=4,
             N=8, new=16, dt=pa.PA_F16)
    a.update(kw)
    ptr = ("bounds", "scales", "kc", "ks", "tables", "first", "lens")
    assert pa.lib.pa_block_bounds(*[ctypes.c_void_p(v) if k in ptr else v for k, v in a.items()], None) == status


def test_model_score_bounds_the_products():
    """The score is not below any product of the query with a key of the block by more than
    the roundings of the codes of q: half a step of s_g per dim times |key| <= 127 steps."""
    rng = np.random.default_rng(0)
    for _ in range(20):
        k = rng.standard_normal((12, BS, 64)).astype(np.float32) + rng.standard_normal(64).astype(np.float32)
        q = rng.standard_normal((3, 64)).astype(np.float32)
        codes, s = M.boxes(k)
        c, sq = M.q_codes(q)
        best = np.einsum("gd,ntd->gnt", q.astype(np.float64), k.astype(np.float64)).max((0, 2))
        slack = 0.5 * sq.max() * np.abs(k).sum(-1).max(-1)
        assert (M.scores(q, codes, s) >= best - slack * (1 + 1e-5)).all()


# ---------------------------------------------------------------------------
def to_dev(x, dtype):
    if dtype == "bfloat16":
        return torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def to_store(x, dtype):
    """fp64 -> the storage dtype (bf16 as uint16 patterns), rounded to nearest even."""
    if dtype == "bfloat16":
        return torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return x.astype(dtype)


def paged(rng, lens, extra=3):
    """Shuffled tables (-1 past a row's blocks) and the pool's size."""
    nb = [-(-max(0, int(n)) // BS) for n in lens]
    N, W = sum(nb) + extra, max(1, max(nb))
    perm = rng.permutation(N).astype(np.int32)
    t = np.full((len(lens), W), -1, np.int32)
    at = 0
    for b, k in enumerate(nb):
        t[b, :k] = perm[at:at + k]
        at += k
    return t, N


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16", "int8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 3, 8])
def test_boxes(dtype, d, H):
    rng = np.random.default_rng(d + H)
    lens, first = [0, 1, 15, 16, 17, 160, 33, 31], [0, 0, 0, 0, 16, 37, 32, 5]
    tables, N = paged(rng, lens)
    x = rng.standard_normal((N, H, BS, d)) * np.exp(rng.uniform(-3, 3, (N, H, 1, 1)))
    ks = None
    if dtype == "int8":
        kc = rng.integers(-127, 128, x.shape).astype(np.int8)
        ks = np.exp(rng.uniform(-5, 1, (N, H))).astype(np.float32)
        keys = (kc.astype(np.float32) * ks[:, :, None, None]).astype(np.float32)
    else:
        kc = to_store(x, dtype)
        keys = M.values(kc)
    for firsts, new in ((first, 130), (None, 160), (first, 123)):
        bounds = torch.full((N, H, 2, d), 55, dtype=torch.int8, device="cuda")
        scales = torch.full((N, H), 7.0, device="cuda")
        pa.pa_get_error_flags(reset=True)
        pa.pa_block_bounds(bounds, scales, to_dev(kc, dtype), to_dev(tables, "i"), to_dev(np.array(lens, np.int32), "i"), new,
                           first_lens=None if firsts is None else to_dev(np.array(firsts, np.int32), "i"),
                           k_scales=None if ks is None else to_dev(ks, "f"))
        assert pa.pa_get_error_flags(reset=True) == 0
        want, ws = np.full((N, H, 2, d), 55, np.int8), np.full((N, H), 7, np.float32)
        codes, s = M.boxes(keys)
        for b, n in enumerate(lens):
            for j in range((firsts[b] if firsts else 0) // BS, n // BS):
                want[tables[b, j]], ws[tables[b, j]] = codes[tables[b, j]], s[tables[b, j]]
        assert np.array_equal(scales.cpu().numpy(), ws)
        assert np.array_equal(bounds.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_boxes_of_odd_values(dtype):
    """Zeros, one value, infinities, NaN, the largest and smallest values of the type."""
    d, H = 64, 1
    big, tiny = float(torch.finfo(TD[dtype]).max), float(torch.finfo(TD[dtype]).tiny)
    tiles = np.zeros((9, H, BS, d))
    tiles[1] = 3.5
    tiles[2, 0, 3, 5] = np.inf
    tiles[3, 0, 15, 63] = np.nan
    tiles[4, 0, 0, 0], tiles[4, 0, 1, 1] = big, -big
    tiles[5, 0, 0, 0], tiles[5, 0, 1, 1] = tiny, -tiny / 2
    tiles[6] = -1.0
    tiles[7, 0, 7, 7] = -np.inf
    tiles[8, 0, :, ::2] = np.nan
    kc = to_store(tiles, dtype)
    codes, s = M.boxes(M.values(kc))
    bounds = torch.zeros((9, H, 2, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((9, H), device="cuda")
    t = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    pa.pa_block_bounds(bounds, scales, to_dev(kc, dtype), t, torch.tensor([144], dtype=torch.int32, device="cuda"), 144)
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(bounds.cpu().numpy(), codes)


@pytest.mark.gpu
def test_boxes_flags():
    kc = torch.ones((4, 2, BS, 64), dtype=torch.float16, device="cuda")
    bounds, scales = torch.zeros((4, 2, 2, 64), dtype=torch.int8, device="cuda"), torch.zeros((4, 2), device="cuda")
    t = torch.tensor([[0, 7, 2], [-1, 1, 3]], dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pa.pa_get_error_flags(reset=True)
    pa.pa_block_bounds(bounds, scales, kc, t, i32(48, 16), 48)
    assert pa.pa_get_error_flags(reset=True) == pa.PA_EFLAG_BAD_BLOCK
    assert (scales[[0, 2]] > 0).all() and (scales[[1, 3]] == 0).all()
    scales.zero_()
    pa.pa_block_bounds(bounds, scales, kc, t, i32(0, 48), 16, first_lens=i32(0, 16))   # grew by two blocks, told of one
    assert pa.pa_get_error_flags(reset=True) == pa.PA_EFLAG_BAD_LENGTH
    assert (scales[1] > 0).all() and (scales[3] == 0).all()
    pa.pa_block_bounds(bounds, scales, kc, t[:1], i32(1 << 30), 48, first_lens=i32(32))  # lengths past the table's width
    assert pa.pa_get_error_flags(reset=True) == 0 and (scales[2] > 0).all()
    pa.pa_block_bounds(bounds, scales, kc, t[:1], i32(-5), 48, first_lens=i32(-5))
    assert pa.pa_get_error_flags(reset=True) == 0


# ---------------------------------------------------------------------------
def run_select(q, dtype, codes, scales, tables, lens, K, sink, recent, max_len, Q=1):
    B, _, Hq, d = q.shape
    H = scales.shape[1]
    lead = (B, Q) if Q > 1 else (B,)
    sel = torch.full(lead + (H, K), 99, dtype=torch.int32, device="cuda")
    cnt = torch.full(lead + (H,), 99, dtype=torch.int32, device="cuda")
    qt = to_dev(q, dtype).reshape(lead + (Hq, d)).contiguous()
    pa.pa_select_blocks(sel, cnt, qt, to_dev(codes, "i"), to_dev(scales, "f"), to_dev(tables, "i"),
                        to_dev(np.array(lens, np.int32), "i"), max_len, sink, recent)
    return sel.cpu().numpy().reshape(B, Q, H, K), cnt.cpu().numpy().reshape(B, Q, H)


def select_case(rng, lens, H, G, d, dtype, Q=1):
    tables, N = paged(rng, lens)
    keys = rng.standard_normal((N, H, BS, d)) * 0.7 + rng.standard_normal((1, H, 1, d))
    codes, scales = M.boxes(M.values(to_store(keys, dtype)))
    q = to_store(rng.standard_normal((len(lens), Q, H * G, d)), dtype)
    return tables, codes, scales, q


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (8, 4), (3, 8), (1, 17), (2, 64)])
def test_choices(dtype, d, H, G):
    rng = np.random.default_rng(d + 10 * H + G)
    lens = [0, 1, 16, 17, 320, 333, 1000, 2047]
    tables, codes, scales, q = select_case(rng, lens, H, G, d, dtype)
    for K, sink, recent in ((1, 0, 1), (20, 1, 2), (21, 5, 5), (33, 0, 33)):
        pa.pa_get_error_flags(reset=True)
        got = run_select(q, dtype, codes, scales, tables, lens, K, sink, recent, 2047)
        want = M.choose(M.values(q), codes, scales, tables, lens, K, sink, recent, 2047)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), (K, sink, recent)
        assert pa.pa_get_error_flags(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("L,K", [(4096 + 5, 64), (32768, 100), (131072, 256), (131072, 1), (524288, 4096)])
def test_choices_of_long_rows(L, K):
    """One to eight CTAs per row; keys of up to 32768 blocks in one CTA's memory."""
    rng = np.random.default_rng(L)
    H, G, d, n = 2, 4, 64, -(-L // BS)
    N = 257
    tables = rng.integers(0, N, (1, n)).astype(np.int32)   # blocks repeat: many equal scores
    tables[0, ::7] = rng.integers(0, 3, len(tables[0, ::7]))
    codes, scales = M.boxes(rng.standard_normal((N, H, BS, d)).astype(np.float32))
    q = rng.standard_normal((1, 1, H * G, d)).astype(np.float16)
    got = run_select(q, "float16", codes, scales, tables, [L], K, 0, 1, L)
    want = M.choose(M.values(q), codes, scales, tables, [L], K, 0, 1, L)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("B,L", [(10, 16 * 1100), (14, 16 * 900), (20, 16 * 390 + 3), (37, 16 * 300), (50, 16 * 300),
                                 (74, 16 * 520)])
def test_choices_at_every_cluster_size(B, L):
    """Two KV heads and B rows: seven, five, three, two and one CTAs per row, of 256 and 512 threads."""
    rng = np.random.default_rng(B)
    H, G, d, n, N, K = 2, 2, 64, -(-L // BS), 300, 30
    tables = rng.integers(0, N, (B, n)).astype(np.int32)
    codes, scales = M.boxes(rng.standard_normal((N, H, BS, d)).astype(np.float32))
    lens = [L - 16 * int(x) for x in rng.integers(0, 40, B)]
    q = to_store(rng.standard_normal((B, 1, H * G, d)), "bfloat16")
    got = run_select(q, "bfloat16", codes, scales, tables, lens, K, 1, 2, L)
    want = M.choose(M.values(q), codes, scales, tables, lens, K, 1, 2, L)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [2, 3])
def test_choices_of_several_new_tokens(Q):
    rng = np.random.default_rng(Q)
    lens = [1, 2, 3, 17, 18, 400, 513]
    tables, codes, scales, q = select_case(rng, lens, 2, 2, 128, "bfloat16", Q)
    got = run_select(q, "bfloat16", codes, scales, tables, lens, 9, 1, 2, 600, Q)
    want = M.choose(M.values(q), codes, scales, tables, lens, 9, 1, 2, 600)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index():
    d, n = 64, 500
    codes, scales = np.zeros((n, 1, 2, d), np.int8), np.ones((n, 1), np.float32)
    codes[100:200] = 3
    codes[300:310] = 7
    tables = np.arange(n, dtype=np.int32)[None]
    q = np.ones((1, 1, 1, d), np.float16)
    for K in (3, 8, 13, 14, 50, 111, 112, 113, 114, 400, 499):
        got, _ = run_select(q, "float16", codes, scales, tables, [n * BS], K, 1, 2, n * BS)
        want, _ = M.choose(M.values(q), codes, scales, tables, [n * BS], K, 1, 2, n * BS)
        assert np.array_equal(got, want), K


@pytest.mark.gpu
def test_odd_scores():
    """Scales of 0, infinity and NaN, scores that overflow or vanish, heads that are zero,
    infinite or NaN, blocks outside the pool."""
    rng = np.random.default_rng(9)
    H, G, d, lens = 1, 4, 64, [700, 700, 700, 640]
    tables, codes, scales, q = select_case(rng, lens, H, G, d, "float32")
    ids = tables[0]
    scales[ids[5]], scales[ids[9]], scales[ids[11]], scales[ids[13]] = np.inf, np.nan, 0, 1e38
    scales[ids[14]], scales[ids[15]] = 1e-44, 3e38
    q[0, 0, 0], q[0, 0, 1, 3], q[1, 0, 2, 0] = 0, np.inf, np.nan
    q[2, 0, :, :] = 0
    q[3, 0] *= 1e37
    for K in (4, 6, 10, 30):
        got = run_select(q, "float32", codes, scales, tables, lens, K, 1, 1, 700)
        want = M.choose(q, codes, np.where(np.isnan(scales), np.float32(np.inf), scales), tables, lens, K, 1, 1, 700)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    tables[0, 6], tables[0, 20] = -1, len(scales)
    pa.pa_get_error_flags(reset=True)
    for K in (10, 42, 43):
        got = run_select(q, "float32", codes, scales, tables, lens, K, 1, 1, 700)
        want = M.choose(q, codes, np.where(np.isnan(scales), np.float32(np.inf), scales), tables, lens, K, 1, 1, 700)
        assert np.array_equal(got[0], want[0])
    assert pa.pa_get_error_flags(reset=True) == pa.PA_EFLAG_BAD_BLOCK


@pytest.mark.gpu
def test_lengths_past_the_bounds_are_cut():
    rng = np.random.default_rng(3)
    lens = [100, 640, 640]
    tables, codes, scales, q = select_case(rng, lens, 1, 1, 64, "float16")
    for given, max_len in (([100, 640, 640], 333), ([-7, 1 << 30, -2147483648], 1 << 19)):
        got = run_select(q, "float16", codes, scales, tables, given, 7, 1, 1, max_len)
        want = M.choose(M.values(q), codes, scales, tables, given, 7, 1, 1, max_len)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("low", ["minus one", "minus infinity", "a bad block", "nothing"])
@pytest.mark.parametrize("n,infs,K", [(60, 20, 13), (700, 600, 13), (700, 512, 13), (700, 513, 515), (9000, 5000, 3000),
                                      (9000, 300, 40)])
def test_more_boxes_that_are_not_finite_than_picks(n, infs, K, low):
    """Every box that is not finite scores +inf, the largest key there is, whose histogram bin ends
    at the top of the keys' 32 bits: with more of them than picks the cut lies in that bin, whatever
    the lowest score of the row makes the bins' width.  The row behind keeps its list."""
    d, N = 64, 64
    rng = np.random.default_rng(n + infs)
    codes, scales = M.boxes(rng.standard_normal((N, 1, BS, d)).astype(np.float32) + np.float32(2))
    scales[:8] = np.inf
    codes[:8] = 0
    tables = rng.integers(8 if low == "nothing" else 9, N, (1, n)).astype(np.int32)
    tables[0, rng.permutation(np.arange(1, n - 2))[:infs]] = rng.integers(0, 8, infs)
    if low in ("minus one", "minus infinity"):
        codes[8], scales[8] = -127, np.float32(1e-3 if low == "minus one" else 1e38)
        tables[0, 5] = 8
    elif low == "a bad block":
        tables[0, 5] = -1
    q = np.ones((1, 1, 2, d), np.float16)
    sel = torch.full((2, 1, K), 99, dtype=torch.int32, device="cuda")
    cnt = torch.full((2, 1), 99, dtype=torch.int32, device="cuda")
    pa.pa_get_error_flags(reset=True)
    pa.pa_select_blocks(sel[:1], cnt[:1], to_dev(q, "float16")[0], to_dev(codes, "i"), to_dev(scales, "f"), to_dev(tables, "i"),
                        torch.tensor([n * BS], dtype=torch.int32, device="cuda"), n * BS, 1, 2)
    assert pa.pa_get_error_flags(reset=True) == (pa.PA_EFLAG_BAD_BLOCK if low == "a bad block" else 0)
    want = M.choose(M.values(q), codes, scales, tables, [n * BS], K, 1, 2, n * BS)
    assert np.array_equal(sel[:1].cpu().numpy(), want[0][0]) and int(cnt[0]) == K
    assert (sel[1] == 99).all() and int(cnt[1]) == 99


def narrowed(keys, need, kl, kh):
    """The picker's narrowing of the cut, in Python's whole numbers with the kernel's 32-bit
    wrap-around: the range it ends with and the keys inside that it expects there."""
    while True:
        sh = max(0, (kh - kl).bit_length() - 8)
        hist = np.bincount((keys[(keys >= kl) & (keys <= kh)] - kl) >> sh, minlength=256)
        assert len(hist) == 256
        above = np.concatenate((np.cumsum(hist[::-1])[::-1][1:], [0]))
        (b,) = np.flatnonzero((above < need) & (above + hist >= need))
        need -= int(above[b])
        kl += int(b) << sh
        kh = (kl + min(kh - kl, (1 << sh) - 1)) & 0xffffffff
        if hist[b] == need or sh == 0 or hist[b] <= 512:
            return kl, kh, int(hist[b])


@pytest.mark.parametrize("low", [0, 0x007fffff, 0x407fffff, 0x7fffffff, 0xff7fffff, 0xff800000])
@pytest.mark.parametrize("infs", [20, 513, 5000])
def test_the_cut_stays_in_range(low, infs):
    """The bin that holds the cut, its end among 32-bit keys, holds the keys that were counted."""
    keys = np.full(infs + 1, 0xff800000, np.int64)
    keys[3] = low
    for need in (1, 10, infs - 1):
        kl, kh, n = narrowed(keys, need, int(keys.min()), int(keys.max()))
        assert kl <= kh and ((keys >= kl) & (keys <= kh)).sum() == n


@pytest.mark.parametrize("kw", [dict(num_seqs=1 << 30, query_len=1 << 30, num_kv_heads=16, num_q_heads=16),
                                dict(num_seqs=(1 << 31) - 1, query_len=(1 << 31) - 1, num_kv_heads=65535, num_q_heads=65535),
                                dict(num_seqs=1 << 27, num_kv_heads=1), dict(num_seqs=1, query_len=1 << 27, num_kv_heads=1),
                                dict(num_seqs=1 << 16, query_len=1 << 16, num_kv_heads=1)])
def test_row_counts_past_the_limit_are_refused(kw):
    """Also where the number of (row, KV head) pairs passes 64 bits, or the rows 32."""
    f = ctypes.c_void_p(FAKE)
    p = sparse_params(**kw)
    assert pa.lib.pa_select_blocks(*[f] * 7, ctypes.byref(p), None) == pa.PA_ERR_UNSUPPORTED
    assert pa.lib.pa_decode_selected(*[f] * 8, 0.1, ctypes.byref(p), None) == pa.PA_ERR_UNSUPPORTED
    assert pa.lib.pa_decode_sparse(*[f] * 10, 0.1, ctypes.byref(p), None) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,H,Q,d,n,K", [("bfloat16", 112, 8, 1, 128, 256, 64), ("float16", 57, 8, 2, 128, 100, 40),
                                               ("float32", 300, 3, 1, 64, 40, 9), ("float16", 223, 4, 1, 256, 130, 7),
                                               ("bfloat16", 112, 8, 1, 64, 512, 200)])
def test_choices_of_very_many_short_rows(dtype, B, H, Q, d, n, K):
    """More than 888 rows of at most 512 blocks: CTAs of 128 threads."""
    rng = np.random.default_rng(B + d)
    G, N = 2, 300
    assert B * Q * H > 6 * 148 and n <= 512
    tables = rng.integers(0, N, (B, n)).astype(np.int32)   # blocks repeat: equal scores
    codes, scales = M.boxes(rng.standard_normal((N, H, BS, d)).astype(np.float32))
    lens = [int(x) for x in rng.integers(1, n * BS + 1, B)]
    lens[3], lens[7] = n * BS, 0
    q = to_store(rng.standard_normal((B, Q, H * G, d)), dtype)
    pa.pa_get_error_flags(reset=True)
    got = run_select(q, dtype, codes, scales, tables, lens, K, 1, 2, n * BS, Q)
    assert pa.pa_get_error_flags(reset=True) == 0
    want = M.choose(M.values(q), codes, scales, tables, lens, K, 1, 2, n * BS)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_boxes_of_odd_int8_scales(d):
    """Scales that are negative, zero, infinite, NaN, very large and very small; code -128."""
    rng = np.random.default_rng(d)
    N = 9
    kc = rng.integers(-127, 128, (N, 1, BS, d)).astype(np.int8)
    kc[1, 0, 3, 5] = kc[0, 0, 1, 1] = -128
    kc[2, 0, 0, 0] = 0
    ks = np.array([-0.25, 0.5, np.inf, np.nan, 0, -3e36, 1e-44, -0.0, -1e-3], np.float32)[:, None]
    with np.errstate(all="ignore"):
        codes, s = M.boxes((kc.astype(np.float32) * ks[:, :, None, None]).astype(np.float32))
    bounds = torch.zeros((N, 1, 2, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((N, 1), device="cuda")
    t = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    pa.pa_block_bounds(bounds, scales, to_dev(kc, "i"), t, torch.tensor([N * BS], dtype=torch.int32, device="cuda"), N * BS,
                       k_scales=to_dev(ks, "f"))
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(bounds.cpu().numpy(), codes)
