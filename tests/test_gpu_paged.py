"""Attention of one new token over the paged cache against the 64-bit oracle.

Bound.  With u = 2^-24: a score is off by (2 D + 16) u times its magnitudes
(products summed in the matrix unit, the scales' products, the cap, the bias), and for
codes by what the query loses: E4M3 2^-25 of the row's largest element times sum |k|
(fp16's smallest step at [1, 2)), INT8 2^-16 of it (half a step of 1 / 32512); a weight by
e^2d - 1 < 3 d relative with d that error plus 2^-21 for the exponential.  Rounding the
weights adds 2^-11 (fp16: codes and fp16 values) or 2^-8 (bf16 values); adding n weighted
values in fp32 2 n u at most, the means of waves and parts 16 u.  All of these are relative to
mean |v| + |o|.  INT8 values are added as code + 128 <= 255 and 128 times the weights is
taken out: 2 n u of 2 max |v| each.  The largest weight is at least 2^6 in fp16, and weights
below fp16's range lose 2^-25 each, next to a value of at most 4 max |v| in the units of
the product: n 2^-29 max |v|.  The store adds half an ulp.
The logarithm of the sum is off by d + 2 n u, by 2^-17 for the logarithm of a sum up to 2^38
and by 2^-22 of itself."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import serving as S
from tests.block_util import DTYPES, assert_within, device, half_ulp, values
from tests.serving_util import ints, numpy_of, random_cache, random_table

pytestmark = pytest.mark.gpu
U = 2.0**-24


def _gpu(q, cache, table, kv_len, ws=None, stream=None, lse=True, **kw):
    o = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    t, n = ints(table), ints(kv_len)
    ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    ws = B.paged_attention_workspace(q, cache, t) if ws is None else ws
    if kw.get("slopes") is not None:
        kw["slopes"] = torch.from_numpy(np.asarray(kw["slopes"], np.float32)).cuda()
    B.paged_attention(q, cache, t, n, o, ws, lse=ls, stream=stream, **kw)
    torch.cuda.synchronize()
    return o, ls


def _check(o, lse, qv, nc, table, kv_len, fmt, kind, what, **kw):
    D = qv.shape[-1]
    kw.setdefault("scale", D ** -0.5)
    if kw.get("slopes") is not None:
        kw["slopes"] = np.asarray(kw["slopes"], np.float32)
    want, mean, weight, seen, ls = S.paged_attention(qv, nc, table, kv_len, **kw)
    k, v, _ = S.dense(nc, table)
    fine = lambda a: np.abs(a[np.isfinite(a)]).max(initial=0.0)
    d = (2 * D + 16) * U * weight + 2.0**-21
    if fmt != "values":
        d = d + (2.0**-16 if fmt == "int8" else 2.0**-25) * np.abs(qv).max(-1) * abs(kw["scale"]) * fine(np.abs(k).sum(-1))
    n = seen[..., None]
    rel = 3 * d[..., None] + (2.0**-8 if fmt == "values" and kind == "bf16" else 2.0**-11) + (2 * n + 16) * U
    e = rel * (mean + np.abs(want)) + (4 * n * U * fine(v) if fmt == "int8" else 0.0)
    if fmt != "values" or kind == "fp16":
        e = e + n * 2.0**-29 * fine(v)
    assert_within(values(o), want, np.where(n > 0, e + half_ulp(np.abs(want) + e, kind), 0.0), what)
    if lse is not None:
        got = values(lse)
        assert np.array_equal(np.isinf(got), seen == 0), what
        some = seen > 0
        off = d + 2 * seen * U + 2.0**-17 + 2.0**-22 * np.abs(np.where(some, ls, 0.0))
        assert_within(got[some], ls[some], off[some], what + " lse")


SHAPES = [  # B, Hq, heads, D, page, pages of a row, lengths (None: drawn)
    (1, 1, 1, 16, 16, 1, [1]), (1, 4, 2, 64, 16, 1, [16]), (2, 8, 1, 128, 16, 3, [17, 48]), (3, 6, 2, 80, 32, 4, [63, 64, 65]),
    (1, 32, 8, 128, 64, 10, [600]), (2, 24, 24, 64, 16, 20, None), (4, 8, 8, 112, 128, 3, [0, 1, 257, 384]),
    (1, 17, 1, 128, 64, 5, [299]), (2, 40, 2, 96, 256, 2, None), (1, 32, 1, 64, 32, 9, [288]), (1, 33, 1, 128, 16, 7, [100]),
    (1, 70, 1, 48, 64, 3, [180]), (1, 5, 1, 128, 64, 40, [2560]), (2, 4, 1, 64, 256, 20, None), (1, 2, 1, 32, 128, 33, [4200]),
    (3, 20, 1, 128, 64, 70, [4480, 1024, 1025])]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("int8", "fp16"), ("fp8", "bf16"), ("fp8", "fp16"),
                                      ("values", "bf16"), ("values", "fp16")])
@pytest.mark.parametrize("mode", ["all", "cap", "slopes", "window", "everything"])
def test_against_oracle(shape, fmt, kind, mode):
    B_, Hq, heads, D, page, T, n = shape
    rng = np.random.default_rng(sum(shape[:6]))
    n = rng.integers(0, T * page + 2, B_) if n is None else n
    cache = random_cache(B_ * T + 1, heads, page, D, fmt, kind, sum(shape[:6]))
    table = random_table(B_, T, B_ * T + 1, 5)
    q, qv = device(1.5 * rng.standard_normal((B_, Hq, D)), kind)
    kw = {}
    if mode in ("cap", "everything"):
        kw["softcap"] = 5.0 if Hq % 2 else 100.0
    if mode in ("slopes", "everything"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq)
    if mode in ("window", "everything"):
        kw["window"] = int(rng.integers(1, T * page))
    o, lse = _gpu(q, cache, table, n, **kw)
    _check(o, lse, qv, numpy_of(cache), table, n, fmt, kind, f"{mode} {shape}", **kw)
    o2, _ = _gpu(q, cache, table, n, lse=False, **kw)
    assert torch.equal(o, o2)                          # the same bits, with or without the sums


@pytest.mark.parametrize("window", [1, 15, 16, 17, 63, 64, 65, 127, 1000, 1023, 1024, 1025, 1100, 2**31 - 1])
@pytest.mark.parametrize("fmt", ["int8", "values"])
def test_windows(window, fmt):
    B_, Hq, heads, D, page, T = 3, 4, 2, 64, 16, 130
    n = [T * page, 1087, 40]
    cache = random_cache(B_ * T, heads, page, D, fmt, "bf16", 31)
    table = random_table(B_, T, B_ * T, 32)
    q, qv = device(np.random.default_rng(33).standard_normal((B_, Hq, D)), "bf16")
    o, lse = _gpu(q, cache, table, n, window=window)
    _check(o, lse, qv, numpy_of(cache), table, n, fmt, "bf16", f"window {window}", window=window)


@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("fp8", "bf16"), ("values", "bf16"), ("values", "fp16")])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 1e4, -1e30])
def test_scales_of_any_sign_and_size(fmt, kind, scale):
    B_, Hq, heads, D, page, T = 2, 6, 2, 64, 32, 5
    cache = random_cache(B_ * T, heads, page, D, fmt, kind, 41)
    table = random_table(B_, T, B_ * T, 42)
    q, qv = device(np.random.default_rng(43).standard_normal((B_, Hq, D)), kind)
    n = [150, 3]
    o, lse = _gpu(q, cache, table, n, scale=scale, lse=abs(scale) < 1e5)
    if abs(scale) < 1e5:
        _check(o, lse, qv, numpy_of(cache), table, n, fmt, kind, f"scale {scale}", scale=scale)
    else:           # the best key alone
        k, v, _ = S.dense(numpy_of(cache), table)
        for b in range(B_):
            for h in range(Hq):
                j = np.argmax(np.sign(scale) * (k[b, :n[b], h // 3] @ qv[b, h]))
                want = v[b, j, h // 3]
                assert_within(values(o)[b, h], want, np.abs(want) * 2.0**-10 + half_ulp(want, kind), "best")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
def test_queries_of_any_magnitude(fmt, kind):
    """Rows whose elements differ by more than fp16 holds, the largest and the smallest, zeros."""
    D, heads, page, T = 64, 1, 16, 4
    cache = random_cache(T, heads, page, D, fmt, kind, 51, gain=0.5)
    rng = np.random.default_rng(52)
    rows = [np.zeros(D), np.r_[1.0, rng.standard_normal(D - 1) * 2.0**-12], rng.standard_normal(D) * 2.0**-14,
            np.r_[60000.0, rng.standard_normal(D - 1)]]
    if kind == "bf16":
        rows += [rng.standard_normal(D) * 2.0**-130, rng.standard_normal(D) * 1e30, np.r_[1e38, np.full(D - 1, -1e30)],
                 rng.standard_normal(D) * np.exp2(rng.integers(-60, 5, D))]
    q, qv = device(np.stack(rows)[None], kind)
    table = random_table(1, T, T, 53)
    for scale in (1.0, 1e-30):
        keep = [i for i, r in enumerate(rows) if np.abs(r).max() * scale < 1e4]      # others: one key, a tie decides
        o, lse = _gpu(q, cache, table, [60], scale=scale)
        _check(o[:, keep], lse[:, keep], qv[:, keep], numpy_of(cache), table, [60], fmt, kind, f"scale {scale}", scale=scale)
        assert np.isfinite(values(o)).all()


@pytest.mark.parametrize("fmt,kind", [("int8", "fp16"), ("fp8", "bf16")])
@pytest.mark.parametrize("low,high", [(2.0**-126, 2.0**-120), (2.0**-100, 2.0**60), (1.0, 2.0**100), (0.0, 0.0)])
def test_value_scales_of_any_magnitude(fmt, kind, low, high):
    """Values whose scales differ by many powers of two, in any order: those that count are the largest."""
    D, page, T = 64, 16, 20
    for order in (1, -1):
        cache = random_cache(T, 2, page, D, fmt, kind, 61)
        s = np.geomspace(low, high, T * page)[::order] if high else np.zeros(T * page)
        cache.v_scale.copy_(torch.from_numpy(s.astype(np.float32)).view(T, 1, page).expand(T, 2, page))
        table = np.arange(T)[None].astype(np.int32)
        q, qv = device(0.3 * np.random.default_rng(62).standard_normal((1, 4, D)), kind)
        o, lse = _gpu(q, cache, table, [T * page])
        want, mean, _, _, _ = S.paged_attention(qv, numpy_of(cache), table, [T * page], D ** -0.5)
        if kind == "fp16" and high > 1.0:              # beyond the type: infinite where the oracle is
            got = values(o)
            assert np.array_equal(np.isinf(got), np.abs(want) >= 65520) and not np.isnan(got).any()
            continue
        _check(o, lse, qv, numpy_of(cache), table, [T * page], fmt, kind, f"{low} {high} {order}")


@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("fp8", "fp16"), ("values", "bf16"), ("values", "fp16")])
def test_hidden_places_may_hold_anything(fmt, kind):
    """Past the length, before the window, in pages that do not exist and in pages of others: NaN, infinities and the
    type's lowest value there change no bit."""
    B_, Hq, heads, D, page, T = 3, 6, 2, 64, 16, 12
    cache = random_cache(B_ * T + 2, heads, page, D, fmt, kind, 71)
    table = random_table(B_, T, B_ * T, 72)
    table[0, 3], table[1, 0], table[2, 5], table[2, 6] = -1, B_ * T + 2, 2**31 - 1, -2**31
    n, window = [T * page - 5, 100, 33], 90
    q, qv = device(np.random.default_rng(73).standard_normal((B_, Hq, D)), kind)
    clean, ls = _gpu(q, cache, table, n, window=window)
    _check(clean, ls, qv, numpy_of(cache), table, n, fmt, kind, "clean", window=window)
    for bad in (float("nan"), float("inf"), -float("inf"), "lowest"):
        x = torch.finfo(DTYPES[kind]).min if bad == "lowest" else bad
        seen = torch.zeros((B_ * T + 2, page), dtype=torch.bool, device="cuda")
        for b in range(B_):
            for j in range(max(0, n[b] - window), n[b]):
                if 0 <= table[b, j // page] < B_ * T + 2:
                    seen[int(table[b, j // page]), j % page] = True
        hide = ~seen[:, None, :, None]
        if fmt == "values":
            k, v = torch.where(hide, x, cache.k), torch.where(hide.transpose(2, 3), x, cache.v)
            dirty = B.KVCache(k.to(DTYPES[kind]).contiguous(), v.to(DTYPES[kind]).contiguous())
        else:
            code = 0x7F if fmt == "fp8" else 0x80      # NaN; -128
            put = lambda t, at: torch.where(at, code, t.view(torch.uint8)).to(torch.uint8).view(t.dtype).contiguous()
            scale = lambda t: torch.where(~seen[:, None], x, t).float().contiguous()
            dirty = B.KVCache(put(cache.k, hide), put(cache.v, hide.transpose(2, 3)), scale(cache.k_scale), scale(cache.v_scale))
        o, ls2 = _gpu(q, dirty, table, n, window=window)
        assert torch.equal(o, clean) and torch.equal(ls, ls2), f"{bad}"


@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("fp8", "fp16"), ("values", "bf16"), ("values", "fp16")])
def test_visible_nan_and_infinities(fmt, kind):
    """A key's NaN makes its rows NaN, a value's its element (a code's scale: the whole vector); other heads and requests
    keep theirs."""
    B_, Hq, heads, D, page, T = 2, 4, 2, 64, 32, 3
    table, n = random_table(B_, T, B_ * T, 82), [90, 61]
    q, _ = device(np.random.default_rng(83).standard_normal((B_, Hq, D)), kind)
    make = lambda: random_cache(B_ * T, heads, page, D, fmt, kind, 81)
    clean = values(_gpu(q, make(), table, n)[0])
    at = (int(table[0, 1]), 1, 7)                      # request 0, position 39, second head
    c = make()
    if fmt == "values":
        c.k[at][5] = float("nan")
    else:
        c.k_scale[at] = float("nan")
    o, lse = (values(t) for t in _gpu(q, c, table, n))
    assert np.isnan(o[0, 2:]).all() and np.array_equal(o[0, :2], clean[0, :2]) and np.array_equal(o[1], clean[1])
    assert np.isnan(lse[0, 2:]).all() and np.isfinite(lse[1]).all()
    c = make()
    if fmt == "values":
        c.v[at[0], 1, 5, 7] = float("inf")
        c.v[at[0], 1, 6, 7] = float("-inf")
        c.v[at[0], 1, 8, 7] = float("nan")
    else:
        c.v_scale[at] = float("nan")
    o = values(_gpu(q, c, table, n)[0])
    assert np.array_equal(o[0, :2], clean[0, :2]) and np.array_equal(o[1], clean[1])
    if fmt == "values":
        rest = np.delete(np.arange(D), [5, 6, 8])
        assert (o[0, 2:, 5] == np.inf).all() and (o[0, 2:, 6] == -np.inf).all() and np.isnan(o[0, 2:, 8]).all()
        assert np.array_equal(o[0, 2:][:, rest], clean[0, 2:][:, rest])
    else:
        assert np.isnan(o[0, 2:]).all()
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[1, 0, 3] = bad
        o = values(_gpu(q2, make(), table, n)[0])
        assert np.isnan(o[1, 0]).all() and np.array_equal(o[1, 1:], clean[1, 1:]) and np.array_equal(o[0], clean[0])


def test_infinite_scores_of_keys_that_point_away():
    """A key of -infinity against a positive query has weight 0."""
    for fmt in ("int8", "values"):
        cache = random_cache(2, 1, 32, 64, fmt, "bf16", 91)
        q, qv = device(np.abs(np.random.default_rng(92).standard_normal((1, 2, 64))) + 0.5, "bf16")
        if fmt == "values":
            cache.k[1, 0, 3] = float("-inf")
        else:
            cache.k[1, 0, 3] = -127
            cache.k_scale[1, 0, 3] = float("inf")
        o, _ = _gpu(q, cache, [[1, 0]], [40])
        nc = numpy_of(cache)
        if fmt == "values":
            nc["k"][1, 0, 3] = 0.0
        else:
            nc["ks"][1, 0, 3] = 0.0
        # the same without that key: a page of another place would do; hide it by the weight it has
        k, v, _ = S.dense(nc, np.array([[1, 0]]))
        z = 64 ** -0.5 * np.einsum("hd,jd->hj", qv[0], k[0, :40, 0])
        z[:, 3] = -np.inf
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want = p @ v[0, :40, 0]
        assert_within(values(o)[0], want, 2.0**-7 * (p @ np.abs(v[0, :40, 0])) + 2.0**-8 * np.abs(want), fmt)


@pytest.mark.parametrize("fmt", ["int8", "values"])
def test_shared_pages_strided_rows_and_one_request_by_itself(fmt):
    """Requests that share their first pages, queries in a QKV output, a table that is part of a larger one; each
    request gives the same bits alone, under the same number of parts."""
    B_, Hq, heads, D, page, T = 5, 8, 2, 128, 32, 6
    cache = random_cache(16, heads, page, D, fmt, "bf16", 101)
    rng = np.random.default_rng(102)
    wide = rng.integers(0, 16, (B_, T + 5)).astype(np.int32)
    wide[:, 2:4] = wide[0, 2:4]
    n = [1, 64, 65, 190, 192]
    qkv, _ = device(rng.standard_normal((B_, Hq + 2 * heads, D + 8)), "bf16")
    q = qkv[:, :Hq, :D]
    t = ints(wide)[:, 2:2 + T]
    out = torch.full((B_, Hq + 3, D + 16), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = B.paged_attention_workspace(q, cache, t)
    B.paged_attention(q, cache, t, ints(n), out[:, 1:Hq + 1, 8:D + 8], ws)
    o = out[:, 1:Hq + 1, 8:D + 8]
    _check(o, None, values(q), numpy_of(cache), wide[:, 2:2 + T], n, fmt, "bf16", "strided")
    out[:, 1:Hq + 1, 8:D + 8] = -7.0
    assert bool((out == -7.0).all())                   # nothing beside it was written
    B.paged_attention(q, cache, t, ints(n), o, ws)
    for b in range(B_):
        one = torch.empty((1, Hq, D), dtype=torch.bfloat16, device="cuda")
        B.paged_attention(q[b:b + 1], cache, t[b:b + 1], ints(n)[b:b + 1], one, B.paged_attention_workspace(q[:1], cache, t[:1]))
        assert torch.equal(one[0], o[b])


def test_pages_past_32_bits():
    """A cache of more than 2^32 bytes of keys: pages from its far end."""
    heads, page, D = 8, 256, 128
    pages = (1 << 32) // (heads * page * D) + 40
    k = torch.zeros((pages, heads, page, D), dtype=torch.int8, device="cuda")
    v = torch.zeros((pages, heads, D, page), dtype=torch.int8, device="cuda")
    ks, vs = (torch.zeros((pages, heads, page), device="cuda") for _ in range(2))
    small = random_cache(40, heads, page, D, "int8", "bf16", 111)
    for big, part in ((k, small.k), (v, small.v), (ks, small.k_scale), (vs, small.v_scale)):
        big[pages - 40:] = part
    q, _ = device(np.random.default_rng(112).standard_normal((2, 32, D)), "bf16")
    table = random_table(2, 20, 40, 113)
    n = [20 * page, 777]
    want, _ = _gpu(q, small, table, n)
    o, _ = _gpu(q, B.KVCache(k, v, ks, vs), table + (pages - 40), n)
    assert torch.equal(o, want)


def test_long_caches_with_a_tail_of_small_weights():
    """2^17 keys of equal weight next to one that outweighs any of them: the tail keeps its bits."""
    page, T, D = 256, 512, 64
    cache = random_cache(T, 1, page, D, "int8", "bf16", 121)
    cache.k.zero_()
    cache.k_scale.fill_(1.0)
    cache.k[0, 0, 5, 0] = 12                           # score 12 against 0: weight 1.6e5 of 1.3e5 others
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    table = np.arange(T)[None].astype(np.int32)
    for n in (T * page, T * page - 77):
        o, lse = _gpu(q, cache, table, [n], scale=1.0)
        _check(o, lse, values(q), numpy_of(cache), table, [n], "int8", "bf16", f"{n}", scale=1.0)


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    cache = random_cache(80, 4, 64, 128, "fp8", "bf16", 131)
    g = np.random.default_rng(132)
    calls = [(device(g.standard_normal((2, 16, 128)), "bf16")[0], random_table(2, 40, 80, s), [2500 - s, 1300 + s]) for s in range(4)]
    want = [_gpu(q, cache, t, n)[0] for q, t, n in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    args = [(q, ints(t), ints(n), torch.empty_like(q), B.paged_attention_workspace(q, cache, ints(t))) for q, t, n in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (q, t, n, o, ws) in zip(streams, args):
            B.paged_attention(q, cache, t, n, o, ws, stream=st)
    torch.cuda.synchronize()
    for w, (_, _, _, o, _) in zip(want, args):
        assert torch.equal(w, o)
