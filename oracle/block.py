"""The operators around the quantized linear layer, in 64 bits (test
infrastructure only): residual sum + RMS norm + FP8 codes, the FP8 linear,
rotary positions with several axes, attention.

Written from the definitions, one step after the other; every function also
returns what a bound on a 16-bit kernel's error needs (sums of magnitudes).
OCP E4M3 ("8-bit Floating Point Specification", OFP8): sign, 4 exponent bits
with bias 7, 3 mantissa bits, no infinities, S.1111.111 = NaN, maximum 448.
"""

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def e4m3_values():
    """The 256 values of E4M3 in code order (NaN at 0x7F and 0xFF)."""
    code = np.arange(256)
    sign = np.where(code & 0x80, -1.0, 1.0)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0**-9, (8 + m) * 2.0**-3 * np.exp2(e - 7.0))
    v = np.where((code & 0x7F) == 0x7F, np.nan, v)
    return sign * v


def e4m3_decode(codes):
    return e4m3_values()[np.asarray(codes, np.uint8)]


def e4m3_encode(x):
    """Codes of the nearest E4M3 values (ties to the even code), |x| <= 448."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]                       # 0 .. 448, increasing, even codes have even mantissas
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def blocks(K):
    return [slice(b, min(b + BLOCK, K)) for b in range(0, K, BLOCK)]


def add_rmsnorm(x, weight, eps, residual=None):
    """(h, y, scales): scales[m, b] = max over block b of |y| / 448."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    s = np.stack([np.abs(y[:, b]).max(1) for b in blocks(h.shape[1])], 1) / E4M3_MAX
    return h, y, s


def fp8_dequant(codes, scales, rows_per_scale):
    v = e4m3_decode(codes)
    rows, K = v.shape
    s = np.asarray(scales, np.float64)
    return v * s[np.arange(rows) // rows_per_scale][:, np.arange(K) // BLOCK]


def fp8_linear(xq, xs, wq, ws, bias=None):
    """(Y, sum of |products|)."""
    x, w = fp8_dequant(xq, xs, 1), fp8_dequant(wq, ws, BLOCK)
    y = x @ w.T
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :]
    return y, np.abs(x) @ np.abs(w).T


def rope_angles(positions, dims, theta, shared):
    """[M, pairs] angles in radians."""
    cols, j, total = [], 0, sum(dims)
    for a, d in enumerate(dims):
        for i in range(d // 2):
            e = 2.0 * j / total if shared else 2.0 * i / d
            cols.append(np.asarray(positions, np.float64)[:, a] * float(theta) ** -e)
            j += 1
    return np.stack(cols, 1)


def rope(x, angles, interleaved):
    """x [M, heads, D]; (y, |a| + |b| of each element's pair, 0 where an element is copied)."""
    x = np.asarray(x, np.float64)
    P = angles.shape[1]
    c, s = np.cos(angles)[:, None, :], np.sin(angles)[:, None, :]
    ia, ib = (np.arange(P) * 2, np.arange(P) * 2 + 1) if interleaved else (np.arange(P), np.arange(P) + P)
    y, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def visible(Sq, Skv, n, causal, prefix, q_doc, k_doc):
    """[Sq, Skv] truth values for one batch entry; n keys in use."""
    j = np.arange(Skv)[None, :]
    pos = n - Sq + np.arange(Sq)[:, None]
    see = np.broadcast_to(j < n, (Sq, Skv)).copy()
    if causal:
        see &= (j <= pos) | (j < prefix)
    if q_doc is not None:
        see &= np.asarray(q_doc)[:, None] == np.asarray(k_doc)[None, :]
    return see


def attention(q, k, v, scale, causal=False, softcap=0.0, slopes=None, kv_len=None, prefix=None, q_doc=None,
              k_doc=None):
    """q [B, Sq, Hq, D], k, v [B, Skv, Hkv, D].  Returns (o, mean |v|, score
    error weight, keys seen): mean |v| = sum_j p_j |v_j|; the score error
    weight is an upper bound of sum_d |q_d k_d| |scale| + 4 |score| + |bias|
    over the row's visible keys."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    o, mean = np.zeros((B, Sq, Hq, D)), np.zeros((B, Sq, Hq, D))
    weight, seen = np.zeros((B, Sq, Hq)), np.zeros((B, Sq, Hq), np.int64)
    for b in range(B):
        n = Skv if kv_len is None else min(max(int(kv_len[b]), 0), Skv)
        see = visible(Sq, Skv, n, causal, 0 if prefix is None else int(prefix[b]),
                      None if q_doc is None else q_doc[b], None if k_doc is None else k_doc[b])
        dist = np.abs(n - Sq + np.arange(Sq)[:, None] - np.arange(Skv)[None, :])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            for i in range(Sq):
                js = np.flatnonzero(see[i])
                seen[b, i, h] = js.size
                if js.size == 0:
                    continue
                qk = k[b, js, g] * q[b, i, h]
                z = scale * qk.sum(1)
                big = abs(scale) * np.abs(qk).sum(1)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    big = big + softcap
                if slopes is not None:
                    bias = float(slopes[h]) * dist[i, js]
                    z, big = z - bias, big + np.abs(bias)
                weight[b, i, h] = (big + 4 * np.abs(z)).max()
                p = np.exp(z - z.max())
                p /= p.sum()
                o[b, i, h] = p @ v[b, js, g]
                mean[b, i, h] = p @ np.abs(v[b, js, g])
    return o, mean, weight, seen
