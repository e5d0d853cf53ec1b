"""Measured cases of block-sparse paged decode and of the device-side step tables.

The operators, as a decode loop uses them:

* ``tables``: one step's block tables, slot map, positions and lengths from the
  requests' lengths (``pa_step_tables``): finished requests give their blocks back,
  the others get the blocks that their new tokens need;
* ``bounds``: the per-(block, KV head) box of the keys, eight bits a side, of the
  blocks that filled up (``pa_block_bounds``);
* ``select``: the blocks each query row and KV head attends to, the best by an upper
  estimate of the query's products with the box (``pa_select_blocks``);
* ``attend``: decode attention over selected blocks (``pa_decode_selected``);
* ``sparse``: select and attend in one call (``pa_decode_sparse``).

``run`` computes the plain form with elementary torch operations, or with ``own``
calls the library.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per block
DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2, "int8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _tables(batch, width, admit, prompt, finish, refs, **more):
    return dict(op="tables", batch=batch, width=width, admit=admit, prompt=prompt, finish=finish, refs=refs, **more)


def _bounds(batch, lo, hi, new, kv, d, dtype, **more):
    return dict(op="bounds", batch=batch, lo=lo, hi=hi, new=new, kv=kv, d=d, dtype=dtype, **more)


def _attn(op, batch, lo, hi, q_len, heads, kv, d, dtype, cache, keep, sink, recent, **more):
    return dict(op=op, batch=batch, lo=lo, hi=hi, q_len=q_len, heads=heads, kv=kv, d=d, dtype=dtype, cache=cache,
                keep=keep, sink=sink, recent=recent, **more)


def listed():
    f, b, s = "float16", "bfloat16", "float32"
    return [
        # one step of the ragged continuous-batching trace: 64 requests, one token each, a few ending
        _tables(64, 264, 0.0, 0, 0.03, False, name="tables_step_b64"),
        # a scheduler's mixed step: a quarter of 1024 requests are prompts, shared prefixes counted
        _tables(1024, 264, 0.25, 4096, 0.06, True, name="tables_mixed_b1024"),
        # the boxes of a whole long-context cache, made once after its prefill (16 x 8192 tokens)
        _bounds(16, 8192, 8192, 8192, 8, 128, f, name="bounds_build_long"),
        # the same after one decode step of the ragged batch: one block in sixteen rows fills up
        _bounds(64, 16, 4097, 1, 8, 128, b, name="bounds_step_b64"),
        # block choice for the ragged batch
        _attn("select", 64, 16, 4097, 1, 32, 8, 128, f, f, 64, 1, 2, name="select_b64"),
        # block choice of one very long request
        _attn("select", 1, 131072, 131072, 1, 32, 8, 128, b, b, 256, 1, 4, name="select_b1_128k"),
        # attention over chosen blocks: the ragged batch; the long batch on an int8 cache; a small fp32 one
        _attn("attend", 64, 16, 4097, 1, 32, 8, 128, f, f, 64, 1, 2, name="attend_b64"),
        _attn("attend", 16, 8192, 8192, 1, 32, 8, 128, f, "int8", 128, 1, 2, name="attend_long_int8"),
        _attn("attend", 3, 5, 1000, 1, 4, 2, 64, s, s, 16, 1, 1, name="attend_tiny_f32"),
        # the whole sparse decode of one layer: one long request alone; two new tokens per
        # request (speculative decoding); 32 query heads on one KV head
        _attn("sparse", 1, 32768, 32768, 1, 32, 8, 128, f, f, 128, 1, 2, name="sparse_b1_32k"),
        _attn("sparse", 64, 512, 4097, 2, 32, 8, 128, b, b, 64, 1, 2, name="sparse_specdec_b64"),
        _attn("sparse", 128, 4096, 4096, 1, 32, 1, 128, f, f, 64, 1, 2, name="sparse_mqa_b128"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "bounds", "select", "attend", "sparse"])
    if op == "tables":
        return _tables(_log(rng, 1, 1024), _log(rng, 4, 264), round(rng.uniform(0, 0.25), 3), _log(rng, 16, 4096),
                       round(rng.uniform(0, 0.1), 3), rng.random() < 0.5)
    dtype = rng.choice(["float16", "bfloat16", "float16", "bfloat16", "float32"])
    kv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    batch = _log(rng, 1, 64)
    size = kv * d * SIZE[dtype]
    tokens = 131072 * 2048 // size                   # tokens of the whole batch
    hi = _log(rng, 17, max(18, min(65536, tokens // batch)))
    lo = rng.choice([1, hi // 2 + 1, hi])
    if op == "bounds":
        return _bounds(batch, lo, hi, rng.choice([1, 2, 17, hi]), kv, d, dtype)
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    cache = "int8" if dtype != "float32" and rng.random() < 0.25 else dtype
    sink, recent, q_len = rng.choice([0, 1, 2]), rng.choice([1, 2, 3]), rng.choice([1, 1, 1, 2, 3])
    keep = min(_log(rng, 4, 256), 3584 * 2048 // (size * batch * q_len)) + sink + recent
    return _attn(op, batch, lo, hi, q_len, kv * group, kv, d, dtype, cache, keep, sink, recent)


def _spread(lo, hi, n):
    return [lo + int((hi - lo) * (i + 0.5) / n) for i in range(n)] if n > 1 else [hi] * n


def _prompts(c):
    """Lengths of the step's admitted prompts."""
    top = c["width"] * BS
    return _spread(16, max(16, min(c["prompt"], top)), round(c["batch"] * c["admit"]))


def _lens(c, rnd):
    """The batch's lengths, spread evenly over [lo, hi], in an order of the seed's."""
    B, lo, hi = c["batch"], c["lo"], c["hi"]
    out = _spread(lo, hi, B)
    if c["op"] == "bounds" and c["new"] < BS:  # one row in sixteen fills a block in a step
        out = [max(BS, n - n % BS) if i % BS == 0 else n for i, n in enumerate(out)]
    rnd.shuffle(out)
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _keys(n, kv, d, dtype, g):
    """Keys as a model's: some channels with a mean of their own, and tokens of a block alike."""
    mean = torch.randn((1, kv, 1, d), generator=g, device="cuda")
    k = torch.empty((n, kv, BS, d), dtype=DT[dtype], device="cuda")
    for i in range(0, n, 4096):
        m = min(4096, n - i)
        block = torch.randn((m, kv, 1, d), generator=g, device="cuda")
        k[i:i + m] = 0.8 * torch.randn((m, kv, BS, d), generator=g, device="cuda") + 0.6 * block + mean
    return k


def _to_int8(x):
    """Symmetric int8 of a cache, one scale per (block, KV head)."""
    a = x.float().abs().amax((2, 3))
    s = a / torch.full_like(a, 127.0)
    q = torch.round(x.float() / s[:, :, None, None].clamp(min=1e-30)).clamp(-127, 127)
    return q.to(torch.int8), s


def _paged(lens, g, spare=3):
    """Block tables of the lengths in a shuffled pool, the pool's size and an unused block."""
    nb = [-(-n // BS) for n in lens]
    N, M = sum(nb) + spare, max(1, max(nb))
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(lens), M), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + nb).cumsum(0)[:-1].cuda()
    j = torch.arange(M, device="cuda")
    has = j < torch.tensor(nb).cuda()[:, None]
    t = torch.where(has, perm[(at[:, None] + j).clamp(max=N - 1)], t)
    return t, N, perm[-1:].long()


def prepare(case, seed):
    c, rnd = case, random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] == "tables":
        B, M = c["batch"], c["width"]
        top = M * BS
        admit, finish = round(B * c["admit"]), round(B * c["finish"])
        rows = [(0, n) for n in _prompts(c)]
        rows += [(rnd.randint(16, top - 1), -1 if i < finish else 1) for i in range(B - admit)]
        rnd.shuffle(rows)
        lens, new = [r[0] for r in rows], [r[1] for r in rows]
        tables, used, _ = _paged(lens, g, 0) if sum(lens) else (torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), 0, None)
        tables = torch.nn.functional.pad(tables, (0, M - tables.shape[1]), value=-1)
        N = B * M
        refs = None
        if c["refs"]:
            refs = torch.zeros(N, dtype=torch.int32, device="cuda")
            refs[:used] = 1
            refs[torch.randperm(max(used, 1), generator=g, device="cuda")[:used // 50]] = 2  # also held by a prefix cache
            part = [b for b in range(B) if lens[b] % BS]  # the last, partly filled blocks belong to one request
            refs[tables[part, [lens[b] // BS for b in part]].long()] = 1
        free = torch.zeros(N, dtype=torch.int32, device="cuda")
        free[:N - used] = used + torch.randperm(N - used, generator=g, device="cuda").to(torch.int32)
        T = sum(_prompts(c)) + B + 64  # the step's token buffer is a little longer than its tokens
        st = dict(c=c, tables=tables, lens=i32(lens), new=i32(new), free=free, count=i32([N - used]), refs=refs, T=T,
                  slots=torch.empty(T, dtype=torch.int64, device="cuda"), pos=torch.empty(T, dtype=torch.int32, device="cuda"),
                  starts=torch.empty(B + 1, dtype=torch.int32, device="cuda"), lens_out=torch.empty(B, dtype=torch.int32, device="cuda"),
                  count_out=torch.empty(1, dtype=torch.int32, device="cuda"))
        return st
    lens = _lens(c, rnd)
    kv, d = c["kv"], c["d"]
    tables, N, unused = _paged(lens, g)
    keys = _keys(N, kv, d, c["dtype"], g)
    st = dict(c=c, tables=tables, lens=i32(lens), max_len=max(lens), k_scales=None, v_scales=None)
    if c["op"] == "bounds":
        first = [max(0, n - c["new"]) for n in lens]
        st.update(kc=keys, first=i32(first), spare=unused, bounds=torch.zeros((N, kv, 2, d), dtype=torch.int8, device="cuda"),
                  bscales=torch.zeros((N, kv), device="cuda"))
        # the blocks that this step completes, in table order
        full = [(b, j) for b in range(len(lens)) for j in range(first[b] // BS, lens[b] // BS)]
        full = full or [(0, 0)]
        st["ids"] = tables[[x for x, _ in full], [y for _, y in full]].long()
        return st
    shape = (c["batch"], c["heads"], d) if c["q_len"] == 1 else (c["batch"], c["q_len"], c["heads"], d)
    st["q"] = torch.randn(shape, generator=g, device="cuda").to(DT[c["dtype"]])
    st["scale"] = d ** -0.5
    st["sel"] = torch.empty(shape[:-2] + (kv, c["keep"]), dtype=torch.int32, device="cuda")
    st["nsel"] = torch.empty(shape[:-2] + (kv,), dtype=torch.int32, device="cuda")
    vals = _keys(N, kv, d, c["dtype"], g) if c["op"] != "select" else None
    if c["cache"] == "int8":
        keys, st["k_scales"] = _to_int8(keys)
        if vals is not None:
            vals, st["v_scales"] = _to_int8(vals)
    st["bounds"], st["bscales"] = _box(_cache_values(keys, st["k_scales"], torch.arange(N, device="cuda")))
    if c["op"] == "select":
        return st
    st.update(kc=keys, vc=vals, out=torch.empty_like(st["q"]))
    if c["op"] == "attend":
        # a choice made before (as by an earlier layer): for each row and KV head some of its
        # blocks, ascending, the newest among them
        L = _row_lens(st["lens"], st["q"])
        n = (L + BS - 1) // BS
        K, M = c["keep"], tables.shape[1]
        r = torch.rand(L.shape + (kv, max(M, K)), generator=g, device="cuda")
        j = torch.arange(max(M, K), device="cuda")
        r = torch.where(j == (n - 1)[..., None, None], -1.0, r).masked_fill(j >= n[..., None, None], 2.0)
        chosen = r.argsort(-1)[..., :K]
        cnt = n.clamp(max=K)[..., None].expand(L.shape + (kv,))
        chosen = torch.where(torch.arange(K, device="cuda") < cnt[..., None], chosen, 1 << 30).sort(-1).values
        chosen = torch.where(chosen < (1 << 30), chosen, -1).to(torch.int32)
        st["sel"] = chosen.reshape(st["sel"].shape).contiguous()
        st["nsel"] = cnt.to(torch.int32).reshape(st["nsel"].shape).contiguous()
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _row_lens(lens, q):
    """Tokens that each query row sees, [B][Q]."""
    Q = q.shape[1] if q.dim() == 4 else 1
    return (lens[:, None].long() - Q + 1 + torch.arange(Q, device=lens.device)).clamp(min=0)


def _plain_tables(s):
    lens, new, T = s["lens"].long(), s["new"].long(), s["T"]
    tables, M = s["tables"].long(), s["tables"].shape[1]
    B, N, dev = lens.numel(), s["free"].numel(), lens.device
    j = torch.arange(M, device=dev)
    old = (lens + BS - 1) // BS
    # finished requests: their blocks go back on the stack, in (row, block) order
    fin = new == -1
    gone = (fin[:, None] & (j < old[:, None])).reshape(-1)
    ids = torch.where(gone, tables.reshape(-1), N)
    if s["refs"] is not None:
        refs = torch.nn.functional.pad(s["refs"].long(), (0, 1))
        refs.index_add_(0, ids, -torch.ones_like(ids))
        at = torch.arange(B * M, device=dev)
        last = torch.full((N + 1,), -1, device=dev).scatter_reduce_(0, ids, at, "amax")
        push = gone & (refs[ids] == 0) & (last[ids] == at)
        refs = refs.clamp(min=0)
    else:
        refs, push = None, gone
    run = push.long().cumsum(0)
    count = s["count"].long()
    free = torch.nn.functional.pad(s["free"].long(), (0, 1))
    free = free.scatter(0, torch.where(push, count + run - 1, N), ids)
    avail = count + run[-1]
    # the others: blocks in order while they last
    tok = new.clamp(min=0)
    end = tok.cumsum(0)
    starts = end - tok
    cand = (new > 0) & (lens + new <= M * BS) & (end <= T)
    if refs is not None:
        part = tables.gather(1, (lens // BS).clamp(max=M - 1)[:, None])[:, 0].clamp(min=0)
        cand &= (lens % BS == 0) | (refs[part] <= 1)
    need = torch.where(cand, (lens + tok + BS - 1) // BS - old, 0)
    upto = need.cumsum(0)
    ok = cand & ((need == 0) | (upto <= avail))
    need = torch.where(ok, need, 0)
    first = upto - torch.where(cand, (lens + tok + BS - 1) // BS - old, 0)
    fresh = (j >= old[:, None]) & (j < (old + need)[:, None])
    nth = first[:, None] + j - old[:, None]
    got = free[(avail - 1 - nth).clamp(0, N)]
    tables = torch.where(fresh, got, tables)
    if refs is not None:
        refs = refs.index_fill(0, torch.where(fresh, got, N).reshape(-1), 1)[:N].to(torch.int32)
    # each token's slot
    t = torch.arange(T, device=dev)
    row = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    live = (t < end[-1]) & ok[row]
    pos = lens[row] + t - starts[row]
    slot = tables.reshape(-1)[(row * M + pos // BS).clamp(max=B * M - 1)] * BS + pos % BS
    out = dict(tables=tables.to(torch.int32), lens=torch.where(fin, 0, torch.where(ok, lens + tok, lens)).to(torch.int32),
               slots=torch.where(live, slot, -1), pos=torch.where(live, pos, -1).to(torch.int32),
               starts=torch.nn.functional.pad(end, (1, 0)).clamp(max=T).to(torch.int32),
               free=free[:N].to(torch.int32), count=(avail - need.sum()).to(torch.int32).reshape(1))
    if refs is not None:
        out["refs"] = refs
    return out


def _cache_values(cache, scales, ids):
    """The cache's tiles of blocks `ids` as fp32 values."""
    x = cache[ids].float()
    return x if scales is None else x * scales[ids][..., None, None]


def _box(keys):
    """The keys' box per (block, KV head): codes [..][2][d] and the scale."""
    lo, hi = keys.amin(-2), keys.amax(-2)
    a = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    s = a / torch.full_like(a, 127.0)
    div = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    zero = (s == 0)[..., None]
    lo = torch.floor(lo / div).clamp(-127, 127).masked_fill(zero, 0)
    hi = torch.ceil(hi / div).clamp(-127, 127).masked_fill(zero, 0)
    return torch.stack((lo, hi), -2).to(torch.int8), s


def _plain_bounds(s):
    B, M = s["tables"].shape
    lens, first = s["lens"].long(), s["first"].long()
    W = -(-s["c"]["new"] // BS)
    j = first[:, None] // BS + torch.arange(W, device=lens.device)
    live = j < lens[:, None] // BS
    ids = s["tables"].gather(1, j.clamp(max=M - 1)).long()
    # what is not complete is computed too, and put in a block that no table holds
    codes, scale = _box(_cache_values(s["kc"], s["k_scales"], ids.clamp(min=0).reshape(-1)))
    put = torch.where(live, ids, s["spare"]).reshape(-1)
    s["bounds"].index_copy_(0, put, codes)
    s["bscales"].index_copy_(0, put, scale)
    return dict(box=s["bounds"][s["ids"]] * s["bscales"][s["ids"]][..., None, None])


def _plain_select(s):
    c, q = s["c"], s["q"]
    L = _row_lens(s["lens"], q)
    B, Q = L.shape
    kv, K, M, d = c["kv"], c["keep"], s["tables"].shape[1], c["d"]
    qf = q.float().reshape(B, Q, kv, -1, d)
    a = qf.abs().amax(-1)
    sq = a / torch.full_like(a, 127.0)
    code = torch.round(qf / torch.where(sq > 0, sq, torch.ones_like(sq))[..., None]).clamp(-127, 127)
    ids = s["tables"].clamp(min=0).long()
    box = s["bounds"][ids].float()                               # [B][M][kv][2][d]
    scale = s["bscales"][ids].permute(0, 2, 1)[:, None, :, None]  # [B][1][kv][1][M]
    # whole numbers below 2^24: exact in fp32 in any order
    dot = torch.einsum("bqhgd,bmhd->bqhgm", code.clamp(max=0), box[..., 0, :])
    dot = dot + torch.einsum("bqhgd,bmhd->bqhgm", code.clamp(min=0), box[..., 1, :])
    score = ((dot * scale) * sq[..., None] + 0.0).amax(3)        # [B][Q][kv][M]
    n = ((L + BS - 1) // BS)[..., None, None]
    j = torch.arange(M, device=q.device)
    kind = ((j < c["sink"]) | (j >= n - c["recent"])).int() + 1
    kind = torch.where(j < n, kind, 0).expand_as(score)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, kind.gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)
    if M < K:
        order = torch.nn.functional.pad(order, (0, K - M))
    cnt = n.clamp(max=K)
    pick = torch.where(torch.arange(K, device=q.device) < cnt, order[..., :K], M).sort(-1).values
    pick = torch.where(pick < M, pick, -1).to(torch.int32)
    cnt = cnt[..., 0].expand(B, Q, kv).to(torch.int32)
    return pick.reshape(s["sel"].shape), cnt.reshape(s["nsel"].shape)


def _plain_attend(s, sel, nsel):
    c, q = s["c"], s["q"]
    L = _row_lens(s["lens"], q)
    B, Q = L.shape
    kv, K, d = c["kv"], c["keep"], c["d"]
    sel, nsel = sel.reshape(B, Q, kv, K).long(), nsel.reshape(B, Q, kv)
    live = torch.arange(K, device=q.device) < nsel[..., None]
    row = torch.arange(B, device=q.device)[:, None, None, None]
    ids = s["tables"].long()[row, sel.clamp(min=0)]
    head = torch.arange(kv, device=q.device)[:, None]

    def tiles(cache, scales):
        x = cache[ids, head].float()                             # [B][Q][kv][K][16][d]
        if scales is not None:
            x = x * scales[ids, head][..., None, None]
        return x.reshape(B, Q, kv, K * BS, d)

    at = (sel[..., None] * BS + torch.arange(BS, device=q.device))
    seen = (live[..., None] & (at < L[:, :, None, None, None])).reshape(B, Q, kv, 1, K * BS)
    qf = q.float().reshape(B, Q, kv, -1, d)
    w = (qf @ tiles(s["kc"], s["k_scales"]).transpose(-1, -2)) * s["scale"]
    w = w.masked_fill(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = w.sum(-1, keepdim=True)
    out = (w @ tiles(s["vc"], s["v_scales"])) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(q.shape).to(q.dtype)


def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        from paged_kv_cache_395_b200 import pa
        if op == "tables":
            refs = None if s["refs"] is None else s["refs"].clone()  # the next pass begins from the same counts
            pa.pa_step_tables(s["tables"], s["lens"], s["new"], s["free"], s["count"], s["slots"], seq_lens_out=s["lens_out"],
                              free_count_out=s["count_out"], positions=s["pos"], row_starts=s["starts"], refcounts=refs)
            out = dict(tables=s["tables"], lens=s["lens_out"], slots=s["slots"], pos=s["pos"], starts=s["starts"], free=s["free"],
                       count=s["count_out"])
            if refs is not None:
                out["refs"] = refs
            return out
        if op == "bounds":
            pa.pa_block_bounds(s["bounds"], s["bscales"], s["kc"], s["tables"], s["lens"], c["new"], first_lens=s["first"])
            return dict(box=s["bounds"][s["ids"]] * s["bscales"][s["ids"]][..., None, None])
        if op == "select":
            pa.pa_select_blocks(s["sel"], s["nsel"], s["q"], s["bounds"], s["bscales"], s["tables"], s["lens"], s["max_len"],
                                sink_blocks=c["sink"], recent_blocks=c["recent"])
            return dict(sel=s["sel"], nsel=s["nsel"])
        if op == "attend":
            pa.pa_decode_selected(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["sel"], s["nsel"], s["scale"],
                                  s["max_len"], k_scales=s["k_scales"], v_scales=s["v_scales"])
            return dict(out=s["out"])
        pa.pa_decode_sparse(s["out"], s["q"], s["kc"], s["vc"], s["bounds"], s["bscales"], s["tables"], s["lens"], s["sel"],
                            s["nsel"], s["scale"], s["max_len"], sink_blocks=c["sink"], recent_blocks=c["recent"],
                            k_scales=s["k_scales"], v_scales=s["v_scales"])
        return dict(out=s["out"], sel=s["sel"], nsel=s["nsel"])
    if op == "tables":
        return _plain_tables(s)
    if op == "bounds":
        return _plain_bounds(s)
    if op == "select":
        sel, nsel = _plain_select(s)
        return dict(sel=sel, nsel=nsel)
    if op == "attend":
        return dict(out=_plain_attend(s, s["sel"], s["nsel"]))
    sel, nsel = _plain_select(s)
    return dict(out=_plain_attend(s, sel, nsel), sel=sel, nsel=nsel)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "tables":
        B, M = c["batch"], c["width"]
        admit, finish = round(B * c["admit"]), round(B * c["finish"])
        step = B - admit - finish
        tokens = sum(_prompts(c)) + B + 64
        blocks = sum(-(-n // BS) for n in _prompts(c)) + step / BS  # handed out
        back = finish * M / 2                                       # given back
        per = 4 + 4 + (4 if c["refs"] else 0)           # table entry, stack entry, count
        return {"bytes": int(16 * B + 12 * tokens + per * (blocks + back)), "flops": 0}
    lens = _lens(c, random.Random(0))
    kv, d = c["kv"], c["d"]
    if c["op"] == "bounds":
        full = sum(n // BS - max(0, n - c["new"]) // BS for n in lens)
        tile = BS * d * SIZE[c["dtype"]]
        return {"bytes": int(full * kv * (tile + 2 * d + 4) + 12 * len(lens)), "flops": 2 * full * kv * BS * d}
    Q, G, K, E = c["q_len"], c["heads"] // c["kv"], c["keep"], SIZE[c["dtype"]]
    blocks = sum(-(-n // BS) for n in lens)              # every block's box is read once
    rows = [max(0, n - Q + 1 + t) for n in lens for t in range(Q)]
    scored = sum(-(-n // BS) for n in rows if -(-n // BS) > K)
    scored_once = sum(-(-n // BS) for n in lens if -(-n // BS) > K)
    qo = len(rows) * c["heads"] * d * E
    lists = len(rows) * kv * 4 * (K + 1)
    tbl = 4 * blocks
    sel_bytes = scored_once * kv * (2 * d + 4) + qo + lists + tbl
    sel_flops = scored * kv * G * 2 * 2 * d
    kept = sum(min(n, K * BS) for n in rows) * kv
    tile = 2 * d * SIZE[c["cache"]]
    # tokens that several rows of a request choose are read once at best: the newest row's share
    once = sum(min(n, K * BS) for n in lens) * kv
    att_bytes = once * tile + 2 * qo + lists + tbl
    att_flops = 4 * kept * G * d
    if c["op"] == "select":
        return {"bytes": int(sel_bytes), "flops": int(sel_flops)}
    if c["op"] == "attend":
        return {"bytes": int(att_bytes), "flops": int(att_flops)}
    return {"bytes": int(sel_bytes - qo + att_bytes - lists - tbl), "flops": int(sel_flops + att_flops)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(c, s, sel, nsel):
    """Attention over the chosen blocks, one query row and KV head at a time."""
    q = s["q"].double().reshape(c["batch"], c["q_len"], c["kv"], -1, c["d"]).cpu()
    tables, lens = s["tables"].cpu().long(), s["lens"].tolist()
    sel = sel.reshape(c["batch"], c["q_len"], c["kv"], -1).cpu().long()
    nsel = nsel.reshape(c["batch"], c["q_len"], c["kv"]).cpu()
    out = torch.zeros(q.shape, dtype=torch.float64)
    for b in range(c["batch"]):
        for t in range(c["q_len"]):
            L = max(0, lens[b] - c["q_len"] + 1 + t)
            for h in range(c["kv"]):
                mine = sel[b, t, h, :int(nsel[b, t, h])]
                if not len(mine):
                    continue
                at = (mine[:, None] * BS + torch.arange(BS)).reshape(-1)
                ids = tables[b, mine].to(s["kc"].device)
                k, v = s["kc"][ids, h].double(), s["vc"][ids, h].double()
                if s["k_scales"] is not None:
                    k = k * s["k_scales"][ids, h].double()[:, None, None]
                    v = v * s["v_scales"][ids, h].double()[:, None, None]
                keep = (at < L).to(k.device)
                k, v = k.reshape(-1, c["d"])[keep], v.reshape(-1, c["d"])[keep]
                w = torch.softmax((k @ q[b, t, h].T.to(k.device)) * s["scale"], 0)
                out[b, t, h] = (w.T @ v).cpu()
    return out.reshape(s["q"].shape)


def _exact_choice(c, s):
    """The chosen blocks, one query row and KV head at a time."""
    B, Q, kv, d, K = c["batch"], c["q_len"], c["kv"], c["d"], c["keep"]
    q = s["q"].double().reshape(B, Q, kv, -1, d)
    lens, tables = s["lens"].tolist(), s["tables"].long()
    sel = torch.full((B, Q, kv, K), -1, dtype=torch.int32)
    nsel = torch.zeros((B, Q, kv), dtype=torch.int32)
    for b in range(B):
        for t in range(Q):
            n = -(-max(0, lens[b] - Q + 1 + t) // BS)
            for h in range(kv):
                nsel[b, t, h] = min(n, K)
                if n <= K:
                    sel[b, t, h, :n] = torch.arange(n)
                    continue
                ids = tables[b, :n]
                sq = (q[b, t, h].abs().amax(-1) / 127).float()
                x = (q[b, t, h] / sq.double()[:, None]).float().round().double()
                lo, hi = s["bounds"][ids, h, 0].double(), s["bounds"][ids, h, 1].double()
                dots = torch.maximum(x[:, None] * lo, x[:, None] * hi).sum(-1)
                one = (dots * s["bscales"][ids, h].double()).float().double()   # the definition's two roundings
                score = (one * sq.double()[:, None]).float().amax(0).cpu().tolist()
                must = {j for j in range(n) if j < c["sink"] or j >= n - c["recent"]}
                rest = sorted((j for j in range(n) if j not in must), key=lambda j: (-score[j], j))
                sel[b, t, h] = torch.tensor(sorted(must | set(rest[:K - len(must)])), dtype=torch.int32)
    return sel.reshape(s["sel"].shape), nsel.reshape(s["nsel"].shape)


def exact(case, seed):
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    if c["op"] == "bounds":
        k = s["kc"][s["ids"]].double()
        lo, hi = k.min(2).values, k.max(2).values
        a = k.abs().amax((2, 3))
        scale = (a / 127).float().double()               # the definition's roundings to fp32
        scale1 = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
        lo = (lo / scale1).float().floor().clamp(-127, 127).double()
        hi = (hi / scale1).float().ceil().clamp(-127, 127).double()
        return dict(box=torch.stack((lo, hi), 2) * scale[..., None, None])
    if c["batch"] * c["q_len"] * c["kv"] > 6000:
        return None
    if c["op"] == "attend":
        return dict(out=_exact_rows(c, s, s["sel"], s["nsel"]))
    sel, nsel = _exact_choice(c, s)
    if c["op"] == "select":
        return dict(sel=sel, nsel=nsel)
    return dict(out=_exact_rows(c, s, sel, nsel), sel=sel, nsel=nsel)
