"""pa_decode_selected and pa_decode_sparse: refusals (CPU); attention over chosen blocks
against the numpy model in 64 bits, the choice of pa_decode_sparse bit for bit, and a
decode loop of all the step's calls (GPU).

Tolerances: |err| <= atol + rtol |ref| of gpu_util.TOL.  fp16: each weight is rounded once
to 11 bits, so the result moves by at most 2^-11 sum_t w_t |v_t| <= 2^-11 max|v| (2.4e-3 for
|v| = 5, about 2^-11 |v| / sqrt(tokens) in earnest), and the output's own rounding by 2^-11
|ref|; bf16: P in two parts (2^-17), its output is checked as fp32 and then for being that
value's rounding; fp32: sums in fp32, exponentials to 2^-22.
"""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_395_b200 import pa
from paged_kv_cache_395_b200.block_manager import BlockManager

from . import sparse_model as M
from .gpu_util import assert_close, bits, check_bf16
from .test_sparse_select import BAD_SPARSE, paged, sparse_params, to_dev, to_store

BS = 16
FAKE = 0x1000


@pytest.mark.parametrize("kw,status", BAD_SPARSE)
def test_refusals(kw, status):
    p = sparse_params(**kw)
    f = ctypes.c_void_p(FAKE)
    assert pa.lib.pa_decode_selected(*[f] * 8, 0.1, ctypes.byref(p), None) == status
    assert pa.lib.pa_decode_sparse(*[f] * 10, 0.1, ctypes.byref(p), None) == status


def test_pointers():
    for fn, n, al in ((pa.lib.pa_decode_selected, 8, (2, 3)), (pa.lib.pa_decode_sparse, 10, (2, 3, 4))):
        p = sparse_params()
        assert fn(*[ctypes.c_void_p(FAKE)] * n, 0.1, None, None) == pa.PA_ERR_NULL
        for i in range(n):
            args = [ctypes.c_void_p(None if k == i else FAKE) for k in range(n)]
            assert fn(*args, 0.1, ctypes.byref(p), None) == pa.PA_ERR_NULL
        for i in al:
            args = [ctypes.c_void_p(FAKE + 8 * (k == i)) for k in range(n)]
            assert fn(*args, 0.1, ctypes.byref(p), None) == pa.PA_ERR_ALIGN
        assert fn(*[None] * n, 0.1, ctypes.byref(sparse_params(num_seqs=0)), None) == pa.PA_OK
        args = [ctypes.c_void_p(FAKE)] * n
        assert fn(*args, 0.1, ctypes.byref(sparse_params(kv_dtype=pa.PA_I8)), None) == pa.PA_ERR_NULL  # no scales
        p = sparse_params(num_blocks=1 << 31, num_kv_heads=2, num_q_heads=2)
        assert fn(*args, 0.1, ctypes.byref(p), None) == pa.PA_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
class Case:
    """A paged cache whose slots past each row's length hold NaN (int8: any code)."""

    def __init__(self, lens, H, G, d, dtype, cache=None, Q=1, seed=0, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.G, self.d, self.dtype, self.Q = lens, H, G, d, dtype, Q
        self.tables, N = paged(rng, lens)
        k = rng.standard_normal((N, H, BS, d)) * 0.8 + rng.standard_normal((1, H, 1, d)) * 0.5
        v = rng.standard_normal((N, H, BS, d))
        self.ks = self.vs = None
        if cache == "int8":
            self.ks = (np.abs(k).max((2, 3)) / 127).astype(np.float32)
            self.vs = (np.abs(v).max((2, 3)) / 127).astype(np.float32)
            self.kc = np.rint(k / self.ks[:, :, None, None]).astype(np.int8)
            self.vc = np.rint(v / self.vs[:, :, None, None]).astype(np.int8)
            self.kf, self.vf = self.kc, self.vc
            keys = (self.kc.astype(np.float32) * self.ks[:, :, None, None]).astype(np.float32)
        else:
            used = np.zeros((N, BS), bool)
            for b, n in enumerate(lens):
                for j in range(-(-max(n, 0) // BS)):
                    used[self.tables[b, j], :min(BS, n - j * BS)] = True
            gone = ~used[:, None, :, None] & np.ones(k.shape, bool)
            k[gone], v[gone] = np.nan, np.nan
            self.kc, self.vc = to_store(k, dtype), to_store(v, dtype)
            self.kf, self.vf = M.values(self.kc), M.values(self.vc)
            keys = self.kf
        self.codes, self.bs = M.boxes(keys)
        self.q = to_store(rng.standard_normal((len(lens), Q, H * G, d)) * q_scale, dtype)
        self.qf = M.values(self.q)
        self.scale, self.max_len = d ** -0.5, max([1] + list(lens))
        lead = (len(lens), Q) if Q > 1 else (len(lens),)
        self.lead = lead
        self.dev = dict(q=to_dev(self.q, dtype).reshape(lead + (H * G, d)).contiguous(),
                        kc=to_dev(self.kc, dtype if cache != "int8" else "i"),
                        vc=to_dev(self.vc, dtype if cache != "int8" else "i"), tables=to_dev(self.tables, "i"),
                        lens=to_dev(np.array(lens, np.int32), "i"), bounds=to_dev(self.codes, "i"), bs=to_dev(self.bs, "f"),
                        ks=None if self.ks is None else to_dev(self.ks, "f"),
                        vs=None if self.vs is None else to_dev(self.vs, "f"))

    def lists(self, K, seed=0, shuffle=False):
        """Random chosen blocks: sel [B][Q][H][K], counts."""
        rng = np.random.default_rng(seed)
        B, H = len(self.lens), self.H
        sel, cnt = np.full((B, self.Q, H, K), -1, np.int32), np.zeros((B, self.Q, H), np.int32)
        L = M.row_lens(self.lens, self.Q, self.max_len)
        for b in range(B):
            for t in range(self.Q):
                n = -(-int(L[b, t]) // BS)
                for h in range(H):
                    k = min(n, K)
                    cnt[b, t, h] = k
                    pick = rng.permutation(n)[:k]
                    if k and n - 1 not in pick:
                        pick[0] = n - 1
                    sel[b, t, h, :k] = pick if shuffle else np.sort(pick)
        return sel, cnt

    def attend(self, sel, cnt, out_f32=False):
        d = self.dev
        K = sel.shape[-1]
        s = torch.from_numpy(sel).cuda().reshape(self.lead + (self.H, K)).contiguous()
        c = torch.from_numpy(cnt).cuda().reshape(self.lead + (self.H,)).contiguous()
        out = torch.full(d["q"].shape, float("nan"), dtype=torch.float32 if out_f32 else d["q"].dtype, device="cuda")
        pa.pa_decode_selected(out, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], s, c, self.scale, self.max_len,
                              k_scales=d["ks"], v_scales=d["vs"])
        return out

    def sparse(self, K, sink, recent, out_f32=False):
        d = self.dev
        s = torch.full(self.lead + (self.H, K), 77, dtype=torch.int32, device="cuda")
        c = torch.full(self.lead + (self.H,), 77, dtype=torch.int32, device="cuda")
        out = torch.full(d["q"].shape, float("nan"), dtype=torch.float32 if out_f32 else d["q"].dtype, device="cuda")
        pa.pa_decode_sparse(out, d["q"], d["kc"], d["vc"], d["bounds"], d["bs"], d["tables"], d["lens"], s, c, self.scale,
                            self.max_len, sink, recent, k_scales=d["ks"], v_scales=d["vs"])
        return out, s.cpu().numpy().reshape(len(self.lens), self.Q, self.H, K), \
            c.cpu().numpy().reshape(len(self.lens), self.Q, self.H)

    def model(self, sel, cnt):
        return M.attend(self.qf, self.kf, self.vf, self.tables, self.lens, sel, cnt, self.scale, self.max_len, self.ks,
                        self.vs)

    def check(self, got, ref, got32=None, what=""):
        ref = ref.reshape(got.shape)
        if self.dtype == "bfloat16":
            check_bf16(got, got32, ref, what)
        else:
            assert_close(got, ref, self.dtype, what)


LENS = [0, 1, 15, 16, 17, 31, 160, 333, 1000]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("bfloat16", None), ("float32", None), ("float16", "int8"),
                                         ("bfloat16", "int8")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,G", [(2, 1), (8, 4), (1, 5), (2, 8), (1, 16), (1, 20), (1, 64)])
def test_attention_over_chosen_blocks(dtype, cache, d, H, G):
    w = Case(LENS, H, G, d, dtype, cache, seed=d + G)
    pa.pa_get_error_flags(reset=True)
    for K, shuffle in ((1, False), (9, True), (63, False)):
        sel, cnt = w.lists(K, K, shuffle)
        w.check(w.attend(sel, cnt), w.model(sel, cnt), w.attend(sel, cnt, True), f"K={K}")
    assert pa.pa_get_error_flags(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("bfloat16", None), ("float32", None), ("float16", "int8")])
@pytest.mark.parametrize("B,L,K,d", [(1, 5000, 300, 128), (1, 5000, 17, 128), (3, 3000, 64, 128), (40, 700, 30, 128),
                                     (1, 40000, 2500, 64), (8, 3000, 150, 64), (11, 2300, 128, 128), (35, 2100, 130, 64)])
def test_rows_split_over_ctas(dtype, cache, B, L, K, d):
    """From one CTA per row to eight, of four and eight warps; more blocks per warp than one batch
    of 32."""
    w = Case([L + 3 * b for b in range(B)], 2, 4, d, dtype, cache, seed=L + B)
    sel, cnt = w.lists(K, 5)
    w.check(w.attend(sel, cnt), w.model(sel, cnt), w.attend(sel, cnt, True))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("bfloat16", None), ("float32", None), ("float16", "int8"),
                                         ("bfloat16", "int8")])
@pytest.mark.parametrize("B,H,G,d", [(50, 2, 4, 128), (50, 2, 4, 64), (90, 1, 16, 128), (100, 1, 32, 64), (90, 1, 20, 128),
                                     (250, 2, 3, 64)])
def test_about_a_row_per_sm_and_many_rows(dtype, cache, B, H, G, d):
    """CTAs of 8 and 12 warps, one per row; many rows in CTAs of 3 or 4."""
    rng = np.random.default_rng(B)
    w = Case([int(x) for x in rng.integers(1, 700, B)], H, G, d, dtype, cache, seed=B + d)
    sel, cnt = w.lists(25, 1)
    w.check(w.attend(sel, cnt), w.model(sel, cnt), w.attend(sel, cnt, True))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("Q", [2, 3])
def test_several_new_tokens(dtype, Q):
    w = Case([1, 2, 3, 16, 17, 18, 19, 450], 2, 3, 128, dtype, Q=Q, seed=Q)
    sel, cnt = w.lists(7, Q)
    w.check(w.attend(sel, cnt), w.model(sel, cnt), w.attend(sel, cnt, True))
    out, s, c = w.sparse(7, 1, 2)
    want = M.choose(w.qf, w.codes, w.bs, w.tables, w.lens, 7, 1, 2, w.max_len)
    assert np.array_equal(s, want[0]) and np.array_equal(c, want[1])
    w.check(out, w.model(s, c), w.sparse(7, 1, 2, True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("bfloat16", None), ("float32", None), ("float16", "int8"),
                                         ("bfloat16", "int8")])
@pytest.mark.parametrize("d,H,G,K", [(128, 8, 4, 16), (64, 2, 8, 5), (256, 2, 2, 20), (128, 1, 32, 12), (128, 3, 7, 70)])
def test_choose_and_attend(dtype, cache, d, H, G, K):
    w = Case([0, 1, 16, 80, 100, 640, 1023], H, G, d, dtype, cache, seed=K)
    out, s, c = w.sparse(K, 1, 2)
    want = M.choose(w.qf, w.codes, w.bs, w.tables, w.lens, K, 1, 2, w.max_len)
    assert np.array_equal(s, want[0]) and np.array_equal(c, want[1])
    w.check(out, w.model(s, c), w.sparse(K, 1, 2, True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("bfloat16", None), ("float32", None), ("float16", "int8")])
def test_all_blocks_is_dense_decode(dtype, cache):
    """With every block chosen the result is pa_decode's, to the two calls' tolerances."""
    w = Case([1, 40, 333, 1000], 4, 4, 128, dtype, cache, seed=2)
    out, s, c = w.sparse(63, 1, 1, True)
    d = w.dev
    dense = torch.empty_like(out)
    pa.pa_decode(dense, d["q"], d["kc"], d["vc"], d["tables"], d["lens"], w.scale, w.max_len, d["ks"], d["vs"])
    tol = 2e-5 if dtype == "float32" else 4e-3
    assert torch.allclose(out, dense, atol=tol, rtol=tol)


@pytest.mark.gpu
def test_sharp_softmax_and_long_lists():
    for dtype in ("float16", "bfloat16", "float32"):
        w = Case([2000, 37], 2, 4, 128, dtype, seed=8, q_scale=8.0)
        sel, cnt = w.lists(125, 3)
        # scores up to |q| |k| d^-1/2 ~ 100: fp32 sums of products of that size are off by up to
        # 128 * 2^-24 * 100 ~ 8e-4 at worst and about 1e-5 in earnest, a relative error of the weights
        got, ref = w.attend(sel, cnt, True).double().cpu().numpy(), w.model(sel, cnt)
        assert np.abs(got - ref.reshape(got.shape)).max() < (5e-3 if dtype != "float32" else 1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("float32", None), ("float16", "int8")])
def test_lists_and_tables_with_bad_entries(dtype, cache):
    """Entries outside the row are skipped, repeated ones count twice, counts outside [0, K]
    are cut, table entries outside the pool are skipped and reported."""
    w = Case([100, 100, 100, 100, 100], 2, 2, 64, dtype, cache, seed=4)
    sel = np.array([[-1, 2, 7, 6], [3, 3, 1, 0], [2147483647, -2147483648, 4, 4], [0, 1, 2, 3], [5, 0, 0, 0]], np.int32)
    sel = np.repeat(sel[:, None, None, :], 2, 2).copy()
    cnt = np.repeat(np.array([4, 3, 3, 99, -5], np.int32)[:, None, None], 2, 2).copy()
    pa.pa_get_error_flags(reset=True)
    got = w.attend(sel, cnt)
    assert pa.pa_get_error_flags(reset=True) == 0
    ref = w.model(sel, np.clip(cnt, 0, 4))
    w.check(got, ref)
    assert (ref[4] == 0).all() and (got[4] == 0).all()
    w.tables[0, 2], w.tables[1, 3], w.tables[3, 0] = -4, len(w.bs), 2147483647
    w.dev["tables"] = to_dev(w.tables, "i")
    got = w.attend(sel, cnt)
    assert pa.pa_get_error_flags(reset=True) == pa.PA_EFLAG_BAD_BLOCK
    w.check(got, w.model(sel, np.clip(cnt, 0, 4)))


@pytest.mark.gpu
def test_unaligned_q_and_out():
    w = Case([100, 333], 2, 4, 128, "float16", seed=6)
    sel, cnt = w.lists(5)
    flat = torch.empty(w.dev["q"].numel() + 1, dtype=torch.float16, device="cuda")
    flat[1:] = w.dev["q"].reshape(-1)
    out = torch.empty(w.dev["q"].numel() + 1, dtype=torch.float16, device="cuda")
    q, o = flat[1:].view(w.dev["q"].shape), out[1:].view(w.dev["q"].shape)
    d = w.dev
    pa.pa_decode_selected(o, q, d["kc"], d["vc"], d["tables"], d["lens"], torch.from_numpy(sel[:, 0]).cuda().contiguous(),
                          torch.from_numpy(cnt[:, 0]).cuda().contiguous(), w.scale, w.max_len)
    assert np.array_equal(bits(o), bits(w.attend(sel, cnt)))


@pytest.mark.gpu
def test_same_result_every_time_and_on_another_stream():
    w = Case([5000, 4000], 2, 4, 128, "bfloat16", seed=7)
    out, s, c = w.sparse(100, 1, 2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(st):
            again, s2, c2 = w.sparse(100, 1, 2)
        st.synchronize()
        assert np.array_equal(bits(out), bits(again)) and np.array_equal(s, s2) and np.array_equal(c, c2)


@pytest.mark.gpu
def test_two_streams_at_once():
    a, b = Case([3000] * 4, 8, 4, 128, "float16", seed=1), Case([2500] * 5, 4, 8, 128, "float16", seed=2)
    ra, rb = a.sparse(60, 1, 2)[0], b.sparse(50, 1, 2)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            outs.append((a.attend, a.sparse(60, 1, 2)[0], ra))
        with torch.cuda.stream(s2):
            outs.append((b.attend, b.sparse(50, 1, 2)[0], rb))
    torch.cuda.synchronize()
    for _, got, ref in outs:
        assert np.array_equal(bits(got), bits(ref))


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_sparse_decode_loop(captured):
    """Tables, append, boxes, choice and attention of a growing batch, eager and as a replayed
    graph, with requests that end and begin: every step against the host's manager and the
    numpy model."""
    B, W, N, H, G, d, K = 6, 12, 120, 2, 4, 64, 5
    rng = np.random.default_rng(21)
    bm = BlockManager(N, free_order=rng.permutation(N))
    ids, nxt, hist = [None] * B, 0, {}
    dt = torch.float16
    kc = torch.full((N, H, BS, d), float("nan"), dtype=dt, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    bounds, bscales = torch.zeros((N, H, 2, d), dtype=torch.int8, device="cuda"), torch.full((N, H), float("nan"), device="cuda")
    tables = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens, before = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    news = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = torch.tensor(bm._free, dtype=torch.int32, device="cuda")
    count = torch.tensor([N], dtype=torch.int32, device="cuda")
    T = 256
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    k, v = torch.zeros((T, H, d), dtype=dt, device="cuda"), torch.zeros((T, H, d), dtype=dt, device="cuda")
    q, out = torch.zeros((B, H * G, d), dtype=dt, device="cuda"), torch.zeros((B, H * G, d), dtype=dt, device="cuda")
    sel, nsel = torch.zeros((B, H, K), dtype=torch.int32, device="cuda"), torch.zeros((B, H), dtype=torch.int32, device="cuda")

    def step():
        before.copy_(lens)
        before.masked_fill_(news < 0, 0)
        pa.pa_step_tables(tables, lens, news, free, count, slots)
        pa.pa_reshape_and_cache(k, v, kc, vc, slots)
        pa.pa_block_bounds(bounds, bscales, kc, tables, lens, W * BS, first_lens=before)
        pa.pa_decode_sparse(out, q, kc, vc, bounds, bscales, tables, lens, sel, nsel, d ** -0.5, W * BS, 1, 2)

    graph = None
    if captured:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()  # no tokens yet: warms up
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
    pa.pa_get_error_flags(reset=True)
    for _ in range(60):
        new = np.zeros(B, np.int32)
        for b in range(B):
            if ids[b] is None:
                new[b] = rng.integers(0, 41)
            elif rng.random() < 0.05 or bm.lens[ids[b]] == W * BS:
                new[b] = -1
            else:
                new[b] = 1
        total = int(np.maximum(new, 0).sum())
        kn, vn = rng.standard_normal((T, H, d)).astype(np.float16), rng.standard_normal((T, H, d)).astype(np.float16)
        qn = rng.standard_normal((B, H * G, d)).astype(np.float16)
        news.copy_(torch.from_numpy(new))
        k.copy_(torch.from_numpy(kn))
        v.copy_(torch.from_numpy(vn))
        q.copy_(torch.from_numpy(qn))
        graph.replay() if captured else step()
        for b in range(B):
            if new[b] == -1:
                bm.free_sequence(ids[b])
                ids[b] = None
        want_slots, at = [], 0
        for b in range(B):
            if new[b] > 0 and ids[b] is None:
                want_slots += bm.add_sequence(nxt, int(new[b])).tolist()
                ids[b], hist[nxt] = nxt, ([], [])
                nxt += 1
            elif new[b] > 0:
                want_slots.append(bm.append_slot(ids[b])[0])
            if new[b] > 0:
                hist[ids[b]][0].append(kn[at:at + new[b]])
                hist[ids[b]][1].append(vn[at:at + new[b]])
                at += int(new[b])
        got_slots = slots.cpu().numpy()
        assert got_slots[:total].tolist() == want_slots and (got_slots[total:] == -1).all()
        sel_h, cnt_h, out_h = sel.cpu().numpy(), nsel.cpu().numpy(), out.double().cpu().numpy()
        for b in range(B):
            n = bm.lens[ids[b]] if ids[b] is not None else 0
            if n == 0:
                assert (out_h[b] == 0).all() and (cnt_h[b] == 0).all()
                continue
            kk, vv = np.concatenate(hist[ids[b]][0]), np.concatenate(hist[ids[b]][1])
            nb = -(-n // BS)
            kp, vp = np.zeros((nb * BS, H, d), np.float32), np.zeros((nb * BS, H, d), np.float32)
            kp[:n], vp[:n] = kk, vv
            kp, vp = [x.reshape(nb, BS, H, d).transpose(0, 2, 1, 3) for x in (kp, vp)]
            codes, s = M.boxes(kp)
            t = np.arange(nb, dtype=np.int32)[None]
            qf = qn[b][None, None].astype(np.float32)
            ws, wc = M.choose(qf, codes, s, t, [n], K, 1, 2, n)
            assert np.array_equal(ws[0, 0], sel_h[b]) and np.array_equal(wc[0, 0], cnt_h[b])
            ref = M.attend(qf, kp, vp, t, [n], ws, wc, d ** -0.5, n)[0, 0]
            assert np.all(np.abs(out_h[b] - ref) <= 2e-3 + 2e-3 * np.abs(ref))
    assert pa.pa_get_error_flags(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_nan_and_infinity_inside_a_row_are_seen(dtype):
    """A NaN key or value of a token that is there shows in its KV head's rows and nowhere else;
    its block's box is not finite, so the block is chosen."""
    w = Case([400, 400, 333], 2, 2, 64, dtype, seed=12)
    for what in ("k", "v"):
        kf, vf = w.kf.copy(), w.vf.copy()
        x = int(w.tables[1, 7])
        (kf if what == "k" else vf)[x, 1, 3, 5] = np.nan
        w.dev["kc"], w.dev["vc"] = to_dev(to_store(kf.astype(np.float64), dtype), dtype), \
            to_dev(to_store(vf.astype(np.float64), dtype), dtype)
        codes, s = M.boxes(kf)
        w.dev["bounds"], w.dev["bs"] = to_dev(codes, "i"), to_dev(s, "f")
        out, sel, cnt = w.sparse(12 if what == "k" else 25, 1, 1, True)
        got = out.cpu().numpy().reshape(3, 2, 2, 64)
        bad = np.isnan(got).reshape(3, 2, -1).any(-1)
        assert bad.tolist() == [[False, False], [False, True], [False, False]], what
        if what == "k":
            assert 7 in sel[1, 0, 1] and np.isnan(got[1, 1]).all()
        else:  # only the value's dim
            assert np.isnan(got[1, 1, :, 5]).all() and not np.isnan(got[1, 1, :, 6]).any()


@pytest.mark.gpu
def test_pool_past_32_bit_offsets():
    """Tiles whose elements lie beyond 2^31 and whose bytes beyond 2^32."""
    H, d, N = 8, 128, 150000          # 2.46e9 elements, 4.9e9 bytes a cache
    kc = torch.zeros((N, H, BS, d), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    lens, n = [300, 77], 19
    rng = np.random.default_rng(3)
    t = np.full((2, n), -1, np.int32)
    ids = N - 1 - rng.permutation(40)[:19 + 5].astype(np.int32)
    t[0], t[1, :5] = ids[:19], ids[19:]
    t[0, 3] = 2
    used = np.unique(t[t >= 0])
    k, v = rng.standard_normal((len(used), H, BS, d)).astype(np.float16), rng.standard_normal((len(used), H, BS, d)).astype(np.float16)
    at = torch.from_numpy(used.astype(np.int64)).cuda()
    # the append writes these slots too
    slots = (at[:, None] * BS + torch.arange(BS, device="cuda")).reshape(-1)
    kt = torch.from_numpy(np.ascontiguousarray(k.transpose(0, 2, 1, 3)).reshape(-1, H, d)).cuda()
    vt = torch.from_numpy(np.ascontiguousarray(v.transpose(0, 2, 1, 3)).reshape(-1, H, d)).cuda()
    pa.pa_reshape_and_cache(kt, vt, kc, vc, slots)
    bounds, bs = torch.zeros((N, H, 2, d), dtype=torch.int8, device="cuda"), torch.zeros((N, H), device="cuda")
    td, ld = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    pa.pa_block_bounds(bounds, bs, kc, td, ld, 300)
    q = rng.standard_normal((2, H * 2, d)).astype(np.float16)
    K = 6
    sel, cnt = torch.zeros((2, H, K), dtype=torch.int32, device="cuda"), torch.zeros((2, H), dtype=torch.int32, device="cuda")
    out = torch.zeros((2, H * 2, d), dtype=torch.float16, device="cuda")
    pa.pa_get_error_flags(reset=True)
    pa.pa_decode_sparse(out, torch.from_numpy(q).cuda(), kc, vc, bounds, bs, td, ld, sel, cnt, d ** -0.5, 304, 1, 2)
    assert pa.pa_get_error_flags(reset=True) == 0
    # the model on a small pool of the same tiles
    where = {int(x): i for i, x in enumerate(used)}
    small = np.array([[where.get(int(x), -1) for x in row] for row in t], np.int32)
    kf, vf = k.astype(np.float32), v.astype(np.float32)
    codes, s = M.boxes(kf)
    qf = q.astype(np.float32)[:, None]
    ws, wc = M.choose(qf, codes, s, small, lens, K, 1, 2, 304)
    assert np.array_equal(sel.cpu().numpy(), ws[:, 0]) and np.array_equal(cnt.cpu().numpy(), wc[:, 0])
    assert_close(out, M.attend(qf, kf, vf, small, lens, ws, wc, d ** -0.5, 304)[:, 0], "float16")


@pytest.mark.gpu
def test_padded_batch_and_rows_behind():
    """Rows of length 0 (a padded batch) give zeros, what lies behind the batch stays."""
    w = Case([200, 0, 64, 0], 2, 4, 128, "float16", seed=3)
    d = w.dev
    big = torch.full((6,) + tuple(d["q"].shape[1:]), 7.0, dtype=torch.float16, device="cuda")
    sel, cnt = torch.full((6, 2, 5), 9, dtype=torch.int32, device="cuda"), torch.full((6, 2), 9, dtype=torch.int32, device="cuda")
    pa.pa_decode_sparse(big[:4], d["q"], d["kc"], d["vc"], d["bounds"], d["bs"], d["tables"], d["lens"], sel[:4], cnt[:4],
                        w.scale, w.max_len)
    assert (big[4:] == 7).all() and (sel[4:] == 9).all() and (cnt[4:] == 9).all()
    assert (big[[1, 3]] == 0).all() and (sel[[1, 3]] == -1).all() and (cnt[[1, 3]] == 0).all()
    assert_close(big[:4], w.model(sel[:4, None].cpu().numpy(), cnt[:4, None].cpu().numpy())[:, 0], "float16")


@pytest.mark.gpu
def test_python_refusals():
    w = Case([100, 50], 2, 4, 64, "float16", seed=1)
    d = w.dev
    sel, cnt = torch.zeros((2, 2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    out = torch.empty_like(d["q"])
    good = dict(out=out, q=d["q"], kc=d["kc"], vc=d["vc"], b=d["bounds"], s=d["bs"], t=d["tables"], l=d["lens"], sel=sel,
                cnt=cnt)

    def call(**kw):
        a = dict(good, **kw)
        pa.pa_decode_sparse(a["out"], a["q"], a["kc"], a["vc"], a["b"], a["s"], a["t"], a["l"], a["sel"], a["cnt"],
                            w.scale, w.max_len)

    call()
    for bad, message in ((dict(out=out.cpu()), "CUDA"), (dict(l=d["lens"].cpu()), "CUDA"), (dict(b=d["bounds"].cpu()), "CUDA"),
                         (dict(l=d["lens"].long()), "int32"), (dict(sel=sel.long()), "int32"),
                         (dict(sel=sel[:, :1]), "selected must"), (dict(cnt=cnt[:1]), "selected must"),
                         (dict(t=d["tables"][:1]), "block_tables must"), (dict(q=d["q"][:, :, ::2], out=out[:, :, ::2]), "caches|contiguous"),
                         (dict(t=d["tables"].t().contiguous().t()), "contiguous"), (dict(out=out[:1]), "out must"),
                         (dict(out=out.bfloat16()), "out must"), (dict(vc=d["vc"].bfloat16()), "caches"),
                         (dict(vc=d["vc"][:1]), "caches"), (dict(b=d["bounds"].float()), "bounds"),
                         (dict(b=d["bounds"][:, :, :1]), "bounds"), (dict(s=d["bs"].half()), "bound_scales")):
        with pytest.raises(ValueError, match=message):
            call(**bad)
    with pytest.raises(pa.PaError) as e:
        pa.pa_decode_sparse(out, d["q"], d["kc"], d["vc"], d["bounds"], d["bs"], d["tables"], d["lens"], sel, cnt, 0.1, 100,
                            sink_blocks=3, recent_blocks=2)
    assert e.value.status == pa.PA_ERR_SHAPE
    with pytest.raises(pa.PaError) as e:
        pa.pa_decode_selected(out, d["q"], d["kc"].to(torch.int8), d["vc"].to(torch.int8), d["tables"], d["lens"], sel, cnt,
                              0.1, 100)
    assert e.value.status == pa.PA_ERR_NULL


@pytest.mark.gpu
def test_two_graphs_and_an_eager_call():
    """Calls captured without a call before them at these sizes, replayed in turn and beside an
    eager one."""
    a, b = Case([777, 1300], 4, 2, 64, "bfloat16", seed=31), Case([3000], 2, 7, 128, "float16", seed=32)
    graphs, outs = [], []
    for w, K in ((a, 11), (b, 40)):
        d = w.dev
        sel, cnt = torch.zeros(w.lead + (w.H, K), dtype=torch.int32, device="cuda"), torch.zeros(w.lead + (w.H,), dtype=torch.int32, device="cuda")
        out = torch.zeros_like(d["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_sparse(out, d["q"], d["kc"], d["vc"], d["bounds"], d["bs"], d["tables"], d["lens"], sel, cnt, w.scale,
                                w.max_len, 1, 2)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g in graphs:
            g.replay()
        eager = a.sparse(11, 1, 2)[0]
    torch.cuda.synchronize()
    assert np.array_equal(bits(outs[0]), bits(eager)) and np.array_equal(bits(outs[1]), bits(b.sparse(40, 1, 2)[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("float16", None), ("float32", None), ("bfloat16", "int8")])
def test_nothing_to_see(dtype, cache):
    """max_seq_len 0, or lengths of 0 and below: zeros and empty lists."""
    w = Case([40, 300], 2, 2, 64, dtype, cache, seed=2)
    for lens, max_len in (([40, 300], 0), ([0, -3], 300), ([-2147483648, 0], 300)):
        w.max_len = max_len
        w.dev["lens"] = to_dev(np.array(lens, np.int32), "i")
        out, sel, cnt = w.sparse(9, 1, 2)
        assert (out == 0).all() and (sel == -1).all() and (cnt == 0).all()
        assert (w.attend(*w.lists(9)) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 20), (256, 3)])
def test_several_new_tokens_on_an_int8_cache(dtype, d, G):
    w = Case([2, 17, 33, 500], 2, G, d, dtype, "int8", Q=2, seed=G)
    out, s, c = w.sparse(8, 1, 2)
    want = M.choose(w.qf, w.codes, w.bs, w.tables, w.lens, 8, 1, 2, w.max_len)
    assert np.array_equal(s, want[0]) and np.array_equal(c, want[1])
    w.check(out, w.model(s, c), w.sparse(8, 1, 2, True)[0])


def test_stall_selftest_refusals():
    f = ctypes.c_void_p(FAKE)

    def call(p, stall_at=0, limit_ns=1000, args=(f,) * 8):
        return pa.lib.pa_decode_selected_stall_selftest(*args, 0.1, ctypes.byref(p), stall_at, limit_ns, None)

    assert call(sparse_params(), stall_at=-1) == pa.PA_ERR_SHAPE
    assert call(sparse_params(), limit_ns=0) == pa.PA_ERR_SHAPE
    assert call(sparse_params(q_dtype=pa.PA_F32, kv_dtype=pa.PA_F32)) == pa.PA_ERR_UNSUPPORTED
    assert call(sparse_params(num_seqs=0)) == pa.PA_OK
    for kw, status in BAD_SPARSE:
        assert call(sparse_params(**kw)) == status
    for i in range(8):
        assert call(sparse_params(), args=tuple(ctypes.c_void_p(None if k == i else FAKE) for k in range(8))) == pa.PA_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache,B,G,d,K", [
    ("float16", None, 3, 4, 128, 200),    # a cluster a row, eight warps a CTA
    ("bfloat16", None, 80, 4, 64, 100),   # 12 warps, one CTA a row
    ("float16", None, 230, 3, 64, 40),    # three warps
    ("bfloat16", None, 2, 20, 128, 90),   # heads on the M side
    ("float16", None, 2, 4, 256, 60),     # one block a step
    ("float16", "int8", 2, 4, 128, 100)])
@pytest.mark.parametrize("stall_at", [0, 1, 2])
def test_wait_timeout_of_a_chosen_block(dtype, cache, B, G, d, K, stall_at):
    """The failure path of the bounded waits, without a fault: one block's copies are left
    unissued.  Every wait ends, the flag is set, the row is NaN (not a result without that block),
    the other rows and the next call are as ever."""
    H = 2
    w = Case([K * BS + 7 * b % 50 for b in range(B)], H, G, d, dtype, cache, seed=B)
    sel, cnt = w.lists(K, 1)
    ref = w.attend(sel, cnt)
    x = w.dev
    s = torch.from_numpy(sel).cuda().reshape(w.lead + (H, K)).contiguous()
    c = torch.from_numpy(cnt).cuda().reshape(w.lead + (H,)).contiguous()
    out = torch.zeros_like(x["q"])
    pa.pa_get_error_flags(reset=True)
    limit_ns = 2_000_000
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    pa.pa_decode_selected_stall_selftest(out, x["q"], x["kc"], x["vc"], x["tables"], x["lens"], s, c, w.scale, w.max_len,
                                         stall_at, limit_ns, k_scales=x["ks"], v_scales=x["vs"])
    t1.record()
    torch.cuda.synchronize()
    # the block's wait, and once more the wait for what is in flight
    assert t0.elapsed_time(t1) >= 2 * limit_ns / 1e6
    assert pa.pa_get_error_flags(reset=True) == pa.PA_EFLAG_WAIT_TIMEOUT
    first = min(G, 16 if d == 256 else 32)  # the heads that run together
    assert torch.isnan(out[0, :first]).all()
    good = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    good[0, :first] = False
    assert np.array_equal(bits(out[good]), bits(ref[good]))
    assert np.array_equal(bits(w.attend(sel, cnt)), bits(ref))
    assert pa.pa_get_error_flags(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("B,H,G,Q", [(60, 8, 4, 1), (75, 6, 7, 1), (30, 8, 4, 2)])
def test_many_rows_of_head_dim_128(dtype, B, H, G, Q):
    """444 and more rows of up to 8 query heads: CTAs of three warps, four on an SM."""
    assert B * Q * H >= 3 * 148
    rng = np.random.default_rng(B)
    w = Case([int(x) for x in rng.integers(Q, 500, B)], H, G, 128, dtype, Q=Q, seed=B + G)
    sel, cnt = w.lists(13, 1)
    w.check(w.attend(sel, cnt), w.model(sel, cnt), w.attend(sel, cnt, True))
