"""The paged key-value cache, attention of single tokens over it, and a block's
gated residual norms, in 64 bits (test infrastructure only).

Written from the definitions in include/svdq.h.  A cache is a dict of numpy
arrays in the library's layout: k [pages, heads, page, D], v [pages, heads, D,
page] (codes as the values they stand for before the scale, or values) and, for
codes, ks, vs [pages, heads, page].
"""

import numpy as np

from oracle import block as O


def encode(x, fmt):
    """(codes, scales) of vectors along the last axis; scales are fp32 numbers."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    odd = ~np.isfinite(x).all(-1)
    top = np.where(odd, 0.0, top)
    with np.errstate(all="ignore"):
        if fmt == "int8":
            s = (top.astype(np.float32) * (np.float32(1) / np.float32(127))).astype(np.float64)
            s = np.where(s < 2.0**-126, 0.0, s)
            c = np.rint(np.where(s[..., None] > 0, x / np.where(s > 0, s, 1.0)[..., None], 0.0))
        else:
            e = np.maximum(np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0)), -126)
            s = np.where(top > 0, 2.0**e, 0.0)
            u = x / np.where(s > 0, s, 1.0)[..., None]
            c = O.e4m3_decode(O.e4m3_encode(np.where(odd[..., None], 0.0, u)))
    return np.where(odd[..., None], 0.0, c), np.where(odd, np.nan, s)


def places(table, entry, position, pages, page):
    """[(token, page, place)] of the tokens that a write does not pass over."""
    B, T = table.shape
    out = []
    for m, p in enumerate(position):
        e = m if entry is None else int(entry[m])
        if 0 <= e < B and 0 <= p < T * page and 0 <= table[e, p // page] < pages:
            out.append((m, int(table[e, p // page]), int(p % page)))
    return out


def write(cache, table, entry, position, k, v, fmt):
    """The cache after a write (a copy)."""
    c = {n: a.copy() for n, a in cache.items()}
    pages, _, page, _ = c["k"].shape
    for m, pg, at in places(table, entry, position, pages, page):
        for n, x in (("k", k[m]), ("v", v[m])):
            x = np.asarray(x, np.float64)
            if fmt != "values":
                x, c[n + "s"][pg, :, at] = encode(x, fmt)
            if n == "k":
                c["k"][pg, :, at] = x
            else:
                c["v"][pg, :, :, at] = x
    return c


def dense(cache, table):
    """(k, v [B, T page, heads, D], there [B, T page]): what each position of a request holds; bad pages hold 0."""
    pages, heads, page, D = cache["k"].shape
    B, T = table.shape
    k, v = np.zeros((B, T * page, heads, D)), np.zeros((B, T * page, heads, D))
    there = np.zeros((B, T * page), bool)
    for b in range(B):
        for t in range(T):
            pg = int(table[b, t])
            if not 0 <= pg < pages:
                continue
            at = slice(t * page, (t + 1) * page)
            there[b, at] = True
            kk, vv = cache["k"][pg], cache["v"][pg].transpose(0, 2, 1)
            if "ks" in cache:
                kk, vv = kk * cache["ks"][pg][..., None], vv * cache["vs"][pg][..., None]
            k[b, at], v[b, at] = kk.transpose(1, 0, 2), vv.transpose(1, 0, 2)
    return k, v, there


def paged_attention(q, cache, table, kv_len, scale, softcap=0.0, window=0, slopes=None):
    """q [B, Hq, D] -> (o, mean |v|, score error weight, keys seen, log sum of exponentials), as oracle.block.attention."""
    k, v, there = dense(cache, table)
    B, N = there.shape
    n = np.clip(np.asarray(kv_len), 0, N)
    j = np.arange(N)[None]
    see = there & (j < n[:, None])
    if window:
        see &= j >= n[:, None] - window
    hidden = np.where(see, 0, 1)
    k, v = np.where(see[..., None, None], k, 0.0), np.where(see[..., None, None], v, 0.0)
    o, mean, weight, seen = O.attention(np.asarray(q)[:, None], k, v, scale, softcap=softcap, slopes=slopes, kv_len=n,
                                        q_doc=np.zeros((B, 1), int), k_doc=hidden)
    lse = np.full(np.asarray(q).shape[:2], -np.inf)
    G = q.shape[1] // k.shape[2]
    for b in range(B):
        js = np.flatnonzero(see[b])
        for h in range(q.shape[1]):
            if js.size:
                z = scale * (k[b, js, h // G] @ np.asarray(q, np.float64)[b, h])
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    z = z - float(slopes[h]) * (n[b] - 1 - js)
                lse[b, h] = z.max() + np.log(np.exp(z - z.max()).sum())
    return o[:, 0], mean[:, 0], weight[:, 0], seen[:, 0], lse


def norm(x, kind, eps):
    x = np.asarray(x, np.float64)
    if kind == "layer":
        x = x - x.mean(1, keepdims=True)
    return x if kind == "none" else x / np.sqrt((x * x).mean(1, keepdims=True) + eps)


def gated_norm(x, residual=None, residual_scale=1.0, post="none", post_weight=None, gate=None, pre="rms", weight=None,
               scale=None, shift=None, entry=None, eps=1e-6):
    """(h, y); gate, scale, shift [E, K], entry [M]."""
    b = norm(x, post, eps)
    if post_weight is not None:
        b = b * post_weight
    if gate is not None:
        b = b * gate[entry]
    h = b if residual is None else residual_scale * np.asarray(residual, np.float64) + b
    y = norm(h, pre, eps)
    if weight is not None:
        y = y * weight
    if scale is not None:
        y = y * (1.0 + scale[entry])
    return h, y if shift is None else y + shift[entry]
