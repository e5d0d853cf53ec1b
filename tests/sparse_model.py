"""The block-sparse operators in numpy (tests only): boxes and choices with the definition's
own fp32 roundings, bit for bit, and attention over chosen blocks in 64 bits."""
import numpy as np

BS = 16
f32 = np.float32


def values(x):
    """A cache or q as fp32 values (bf16 as uint16 patterns)."""
    return (x.astype(np.uint32) << 16).view(f32) if x.dtype == np.uint16 else x.astype(f32)


def boxes(keys):
    """keys fp32 [..][16][d] -> int8 codes [..][2][d] and fp32 scales [..]."""
    with np.errstate(all="ignore"):
        lo, hi = keys.min(-2), keys.max(-2)
        a = np.maximum(np.abs(lo), np.abs(hi)).max(-1)
        fin = np.isfinite(a)
        s = np.where(fin, a / f32(127), f32(np.inf)).astype(f32)
        ok = (fin & (s > 0))[..., None]
        div = np.where(ok, s[..., None], f32(1))
        code = np.stack((np.floor((lo / div).astype(f32)), np.ceil((hi / div).astype(f32))), -2)
        code = np.where(ok[..., None, :], np.clip(code, -127, 127), 0)
    return code.astype(np.int8), s


def q_codes(q):
    """q fp32 [..][d] -> int codes and the scale."""
    with np.errstate(all="ignore"):
        s = (np.abs(q).max(-1) / f32(127)).astype(f32)
        s = np.where(np.isfinite(s), s, f32(0))
        div = np.where(s > 0, s, f32(1))[..., None]
        c = np.where(s[..., None] > 0, np.clip(np.rint((q / div).astype(f32)), -127, 127), 0)
    return c.astype(np.int64), s


def row_lens(lens, Q, max_len):
    L = np.minimum(np.maximum(np.asarray(lens, np.int64), 0), max_len)
    return np.maximum(L[:, None] - Q + 1 + np.arange(Q), 0)


def scores(q, codes, scales):
    """q fp32 [G][d], codes int8 [n][2][d], scales fp32 [n] -> fp32 [n]."""
    c, s = q_codes(q)
    lo, hi = codes[:, 0].astype(np.int64), codes[:, 1].astype(np.int64)
    dot = np.maximum(c[:, None] * lo, c[:, None] * hi).sum(-1)
    with np.errstate(all="ignore"):
        one = (dot.astype(f32) * scales).astype(f32)
        sc = (one * s[:, None]).astype(f32).max(0)
    return np.where(np.isfinite(scales), sc, f32(np.inf))


def choose(q, codes, scales, tables, lens, K, sink, recent, max_len):
    """q fp32 [B][Q][Hq][d] -> selected [B][Q][H][K], counts [B][Q][H]."""
    B, Q, Hq, _ = q.shape
    N, H = scales.shape
    G = Hq // H
    sel = np.full((B, Q, H, K), -1, np.int32)
    cnt = np.zeros((B, Q, H), np.int32)
    L = row_lens(lens, Q, min(max_len, tables.shape[1] * BS))
    for b in range(B):
        for t in range(Q):
            n = -(-int(L[b, t]) // BS)
            for h in range(H):
                cnt[b, t, h] = min(n, K)
                if n <= K:
                    sel[b, t, h, :n] = np.arange(n)
                    continue
                ids = tables[b, :n]
                ok = (ids >= 0) & (ids < N)
                at = np.where(ok, ids, 0)
                sc = np.where(ok, scores(q[b, t, h * G:(h + 1) * G], codes[at, h], scales[at, h]).astype(np.float64),
                              -np.inf)
                must = [j for j in range(n) if j < sink or j >= n - recent]
                rest = sorted((j for j in range(n) if not (j < sink or j >= n - recent)), key=lambda j: (-sc[j], j))
                sel[b, t, h] = np.sort(np.array(must + rest[:K - len(must)], np.int32))
    return sel, cnt


def attend(q, kc, vc, tables, lens, sel, cnt, scale, max_len, k_scales=None, v_scales=None):
    """fp64 [B][Q][Hq][d]: softmax attention over the tokens of the listed blocks.  kc, vc
    fp32 (or int8) [N][H][16][d]."""
    B, Q, Hq, d = q.shape
    N, H = kc.shape[:2]
    G = Hq // H
    L = row_lens(lens, Q, min(max_len, tables.shape[1] * BS))
    out = np.zeros((B, Q, Hq, d))
    for b in range(B):
        for t in range(Q):
            for h in range(H):
                ks, vs = [], []
                for j in sel[b, t, h, :max(0, int(cnt[b, t, h]))]:
                    j = int(j)
                    if not 0 <= j * BS < L[b, t]:
                        continue
                    x = int(tables[b, j])
                    if not 0 <= x < N:
                        continue
                    m = min(BS, int(L[b, t]) - j * BS)
                    k, v = kc[x, h, :m].astype(np.float64), vc[x, h, :m].astype(np.float64)
                    ks.append(k if k_scales is None else k * float(k_scales[x, h]))
                    vs.append(v if v_scales is None else v * float(v_scales[x, h]))
                if not ks:
                    continue
                k, v = np.concatenate(ks), np.concatenate(vs)
                for g in range(h * G, (h + 1) * G):
                    s = (k @ q[b, t, g].astype(np.float64)) * scale
                    w = np.exp(s - s.max())
                    out[b, t, g] = (w / w.sum()) @ v
    return out
