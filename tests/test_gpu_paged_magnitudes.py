"""Attention over pages, mostly of 8 bits, where scales, queries and values are of very different size, against the
64-bit oracle.

Bound.  With u = 2^-24, p a key's weight of sum 1, V its largest |v| and n the keys seen:
  score   (2 D + 16) u times its magnitudes, and what the query loses: E4M3 2^-25 of the row's largest element (half of
          fp16's smallest step at [1, 2)), INT8 half a step of 2^-22 of a power of two that the largest is at least
          0.996 of, 2^-22.9 of the largest, each times sum |k|;
  weight  e^2d - 1 < 3 d relative, d that error and 2^-21 for the exponential, on mean |v| + |o|;
  to 16 bits 2^-11 of each term (bf16 values 2^-8), and over codes 2^-25 absolute where the largest product
          p V / (127 or 224) is held above 2^6: 2^-31 of it a key, times codes of at most 127 or 448: n 2^-30 max (p V);
  sums    (2 n + 16) u of mean |v| + |o|; INT8 values are summed as code + 128 <= 255 and 128 times the weights taken out:
          2 n u of at most 3 sum p V.
The store adds half an ulp.  The logarithm of the sum is off by d + 2 n u, 2^-17 and 2^-22 of itself."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import serving as S
from tests.block_util import assert_within, device, half_ulp, values
from tests.serving_util import ints, numpy_of, random_cache, random_table

pytestmark = pytest.mark.gpu
U = 2.0**-24


def _gpu(q, cache, table, kv_len, **kw):
    o = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    t = ints(table)
    B.paged_attention(q, cache, t, ints(kv_len), o, B.paged_attention_workspace(q, cache, t), lse=lse, **kw)
    torch.cuda.synchronize()
    return o, lse


def _bounds(qv, nc, table, kv_len, fmt, scale, exact=False):
    """(o, its bound before the store, log sum, its bound); exact: queries whose elements are multiples of those steps"""
    D = qv.shape[-1]
    want, mean, weight, seen, ls = S.paged_attention(qv, nc, table, kv_len, scale)
    k, v, _ = S.dense(nc, table)
    G = qv.shape[1] // k.shape[2]
    most, total = np.zeros(qv.shape[:2]), np.zeros(qv.shape[:2])      # max and sum of p V
    for b in range(qv.shape[0]):
        for h in range(qv.shape[1]):
            z = scale * (k[b, :kv_len[b], h // G] @ qv[b, h])
            pv = np.exp(z - ls[b, h]) * np.abs(v[b, :kv_len[b], h // G]).max(-1)
            most[b, h], total[b, h] = pv.max(), pv.sum()
    lost = 0.0 if exact or fmt == "values" else 2.0**-22.9 if fmt == "int8" else 2.0**-25
    d = (2 * D + 16) * U * weight + 2.0**-21 + lost * np.abs(qv).max(-1) * abs(scale) * np.abs(k).sum(-1).max()
    n = seen[..., None]
    e = (3 * d[..., None] + (2.0**-8 if fmt == "values" else 2.0**-11) + (2 * n + 16) * U) * (mean + np.abs(want))
    if fmt != "values":
        e = e + n * 2.0**-30 * most[..., None]
    if fmt == "int8":
        e = e + 6 * n * U * total[..., None]
    return want, e, ls, d + 2 * seen * U + 2.0**-17 + 2.0**-22 * np.abs(ls)


def _check(o, lse, qv, cache, table, kv_len, fmt, kind, scale, what, exact=False):
    want, e, ls, off = _bounds(qv, numpy_of(cache), table, kv_len, fmt, scale, exact)
    assert_within(values(o), want, e + half_ulp(np.abs(want) + e, kind), what)
    assert_within(values(lse), ls, off, what + " lse")


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("low,high", [(2.0**103, 2.0**103), (2.0**118, 2.0**118), (2.0**90, 2.0**119), (2.0**-100, 2.0**119)])
@pytest.mark.parametrize("order", [1, -1])
def test_values_near_the_end_of_the_type(fmt, low, high, order):
    """bf16 values of up to 1e38, some elements zero in all of them; in fp16 they are infinite."""
    D, page, T = 64, 16, 20
    for kind in ("bf16", "fp16"):
        cache = random_cache(T, 2, page, D, fmt, kind, 201)
        cache.v.view(torch.uint8)[:, :, 5:9] = 0
        s = np.geomspace(low, high, T * page)[::order] * (1.0 if fmt == "int8" else 127 / 448)
        cache.v_scale.copy_(torch.from_numpy(s.astype(np.float32)).view(T, 1, page).expand(T, 2, page))
        table = np.arange(T)[None].astype(np.int32)
        q, qv = device(0.3 * np.random.default_rng(202).standard_normal((1, 4, D)), kind)
        o, lse = _gpu(q, cache, table, [T * page])
        if kind == "bf16":
            _check(o, lse, qv, cache, table, [T * page], fmt, kind, D ** -0.5, f"{low} {high}")
        else:
            want, e, _, _ = _bounds(qv, numpy_of(cache), table, [T * page], fmt, D ** -0.5)
            got = values(o)
            assert not np.isnan(got).any() and np.isinf(got[np.abs(want) - e >= 65520]).all()
            assert fmt == "int8" or (got[want == 0] == 0).all()      # (INT8: a difference of sums)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
def test_values_near_the_end_of_the_type_in_parts(fmt):
    """Enough keys that blocks share them and their means are joined."""
    D, page, T = 64, 64, 64
    cache = random_cache(T, 2, page, D, fmt, "bf16", 205)
    if fmt == "values":
        cache.v.uniform_(-1e38, 1e38)
    else:
        cache.v_scale.fill_(2.0**118)
    table = random_table(1, T, T, 206)
    q, qv = device(np.random.default_rng(207).standard_normal((1, 4, D)), "bf16")
    assert B.paged_attention_workspace_bytes(cache, 1, T, 4) > 0
    for n in (T * page, 1000):
        o, lse = _gpu(q, cache, table, [n])
        _check(o, lse, qv, cache, table, [n], fmt, "bf16", D ** -0.5, f"{fmt} {n}")


@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
def test_sums_of_many_large_values(fmt):
    """32768 keys to a wave, all of like weight after a first tile of less, every value the same near the end of bf16: the
    output is that value, off by the weights' rounding (2^-8 at most for bf16), the sums' and the store's."""
    D, page, T, requests = 64, 256, 512, 64
    cache = random_cache(T, 8, page, D, fmt, "bf16", 208)
    cache.k.view(torch.uint8).zero_()
    cache.k[:, :, :, 0] = torch.full((T, 8, page), 4.0, device="cuda").to(cache.k.dtype)
    cache.k[:2, :, :, 0] = torch.full((2, 8, page), -1.0, device="cuda").to(cache.k.dtype)      # weight e^-5, 2^-7.2
    if fmt == "values":
        cache.v.fill_(1e38)
        v = float(cache.v[0, 0, 0, 0])
    else:
        cache.k_scale.fill_(1.0)
        cache.v.copy_(torch.full(cache.v.shape, 112.0).to(cache.v.dtype))
        cache.v_scale.fill_(2.0**119)
        v = 112.0 * 2.0**119
    q = torch.zeros((requests, 8, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    table = np.tile(np.arange(T), (requests, 1))       # the requests share their pages
    assert B.paged_attention_workspace_bytes(cache, requests, T, 8) == 0
    o, _ = _gpu(q, cache, table, [T * page] * requests, scale=1.0)
    e = v * (2.0**-8 + (2 * T * page + 16) * U * (3 if fmt == "int8" else 1))
    assert_within(values(o), np.full(q.shape, v), e + half_ulp(np.full(q.shape, v), "bf16"), fmt)


def test_large_values_written_by_the_writer():
    """Values of 1e34 to 1e38 through the whole path."""
    rng = np.random.default_rng(203)
    k, _ = device(rng.standard_normal((100, 2, 64)), "bf16")
    v, _ = device(rng.uniform(-1, 1, (100, 2, 64)) * 10.0 ** rng.uniform(34, 38, (100, 2, 1)) * (np.arange(64) % 9 > 0), "bf16")
    q, qv = device(rng.standard_normal((1, 8, 64)), "bf16")
    table = random_table(1, 4, 4, 204)
    for fmt in ("int8", "fp8"):
        cache = B.KVCache.empty(4, 2, 64, page=32, format=fmt)
        B.cache_write(cache, ints(table), ints(np.arange(100)), k, v, entry=ints(np.zeros(100)))
        o, lse = _gpu(q, cache, table, [100])
        _check(o, lse, qv, cache, table, [100], fmt, "bf16", 0.125, fmt)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("power", [-125, -118, -100, -30, -18, -9, 9, 18, 30, 100, 118])
def test_large_keys_and_small_queries_and_the_other_way_round(fmt, power):
    """Scores of ordinary size whose factors are near the ends of fp32."""
    D, page, T = 64, 32, 5
    cache = random_cache(T, 2, page, D, fmt, "bf16", 211)
    for s in (cache.k_scale, cache.v_scale):
        s.clamp_(min=2.0**-6, max=2.0**-4)
    cache.k_scale.mul_(2.0**-power)
    q, qv = device(np.random.default_rng(212).standard_normal((1, 6, D)) * 2.0**power, "bf16")
    table = random_table(1, T, T, 213)
    o, lse = _gpu(q, cache, table, [150])
    _check(o, lse, qv, cache, table, [150], fmt, "bf16", D ** -0.5, f"2^{power}")


def _laid(z, s, fmt, kind, seed):
    """A cache of one head whose key j scores z[j] against the first unit vector and has value scale s[j]."""
    D, page = 64, 32
    T = -(-len(z) // page)
    cache = random_cache(T, 1, page, D, fmt, kind, seed)
    cache.k.view(torch.uint8).zero_()
    cache.k_scale.fill_(1.0)
    put = lambda a: torch.from_numpy(np.resize(a, T * page).astype(np.float32)).view(T, 1, page).cuda()
    cache.k.view(torch.uint8)[:, :, :, 0] = put(z).to(cache.k.dtype).view(torch.uint8)
    cache.v_scale.copy_(put(s))
    q = torch.zeros((1, 3, D), dtype=torch.bfloat16 if kind == "bf16" else torch.float16, device="cuda")
    q[0, :, 0] = torch.tensor([1.0, 0.5, 0.25])
    return cache, q, np.arange(T)[None].astype(np.int32)


@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("int8", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")])
@pytest.mark.parametrize("gap", [8, 20, 24, 31, 60])
@pytest.mark.parametrize("n", [40, 600, 2100])
def test_large_values_of_little_weight(fmt, kind, gap, n):
    """A few keys of next to no weight have values 2^gap times the others': the others keep their bits, wherever it lies."""
    rng = np.random.default_rng(gap)
    for at in (0, 17, n // 2, n - 1):
        z, s = rng.integers(-2, 3, n).astype(float), rng.uniform(0.5, 1.0, n) * 2.0**-10
        z[at], s[at] = -100.0 * (1 if gap > 8 else 0.5), 2.0**(gap - 10)
        if fmt == "fp8":
            z[at] = -96.0
            s = np.exp2(np.round(np.log2(s)))
        cache, q, table = _laid(z, s, fmt, kind, 221)
        q = q[:, :2]
        o, lse = _gpu(q, cache, table, [n], scale=1.0)
        _check(o, lse, values(q), cache, table, [n], fmt, kind, 1.0, f"gap {gap} at {at}")


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("n", [64, 500, 3000])
def test_products_of_weight_and_value_of_one_size(fmt, order, n):
    """Weights and values' scales each over many powers of two, their products of like size: all of them count."""
    z = np.linspace(-36, 36, n).round()
    if fmt == "fp8":
        z = 4 * (z / 4).round()                        # E4M3 holds these
    s = np.exp2(np.round(-z * 1.4427))
    i = {"rising": slice(None), "falling": slice(None, None, -1), "mixed": np.random.default_rng(222).permutation(n)}[order]
    cache, q, table = _laid(z[i], s[i], fmt, "bf16", 223)
    o, lse = _gpu(q, cache, table, [n], scale=1.0)
    _check(o, lse, values(q), cache, table, [n], fmt, "bf16", 1.0, order)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("ratio", [1, 300, 3000, 30000])
@pytest.mark.parametrize("heads", [6, 20])
def test_query_channels_that_stand_out(fmt, kind, ratio, heads):
    """One channel of the queries is many times the others', and the keys are small there in proportion: the scores come
    from the others, and so do the output's bits.  Multiples of 1 / 64 below 4: 2^-22 of 2^16."""
    D, page, T = 128, 64, 9
    cache = random_cache(T, 1, page, D, fmt, kind, 231)
    cache.k.view(torch.uint8)[..., 77] = 0
    q = np.clip(np.round(np.random.default_rng(232).standard_normal((1, heads, D)) * 64) / 64, -3.5, 3.5)
    q[..., 77] = ratio * np.where(q[..., 77] < 0, -1.9, 1.99)
    q, qv = device(q, kind)
    table = random_table(1, T, T, 233)
    o, lse = _gpu(q, cache, table, [T * page - 3], scale=0.5)
    _check(o, lse, qv, cache, table, [T * page - 3], fmt, kind, 0.5, f"ratio {ratio}", exact=True)
