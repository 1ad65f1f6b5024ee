"""Attention where K, V and Q hold NaN and infinities at keys that some
queries see and others do not.

What a row sees decides: an infinity in V makes its own column that infinity
(both signs: NaN), a NaN in V its column NaN, a NaN in a K or Q row the whole
row; every other output is, to the bit, that of inputs which hold zeros in the odd
places, and those are within the bound of tests/test_gpu_block_attention.py."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import assert_within, values
from tests.test_gpu_block_attention import _bound, _gpu, _make

pytestmark = pytest.mark.gpu

# B, Sq, Skv, Hq, Hkv, D, parts: single tokens, few rows, blocks of 128 rows; keys of one block and shared by several
SHAPES = [(2, 1, 70, 4, 2, 64, False), (1, 1, 5000, 8, 2, 128, True), (3, 5, 5000, 6, 1, 64, True),
          (2, 40, 300, 6, 2, 72, False), (7, 129, 257, 8, 8, 128, False), (13, 129, 131, 8, 8, 64, False),
          (6, 129, 200, 16, 8, 104, False), (1, 700, 2100, 4, 4, 64, True), (1, 330, 2100, 8, 2, 128, True),
          (1, 330, 2100, 8, 2, 104, True)]
ODD = [float("nan"), float("inf"), float("-inf")]


def _arguments(shape, mode):
    B_, Sq, Skv = shape[:3]
    rng = np.random.default_rng(sum(shape[:6]))
    if mode == "causal":
        return dict(causal=True)
    if mode == "lengths":
        return dict(kv_len=rng.integers(Skv // 2, Skv + 1, B_), causal=Sq > 1, prefix=rng.integers(0, Skv // 3, B_))
    if mode == "documents":
        return dict(k_doc=np.sort(rng.integers(0, 4, (B_, Skv)), axis=1), q_doc=rng.integers(0, 4, (B_, Sq)))
    return {}


def _visible(shape, kw):
    B_, Sq, Skv = shape[:3]
    at = lambda n, b: None if kw.get(n) is None else kw[n][b]
    return np.stack([O.visible(Sq, Skv, Skv if kw.get("kv_len") is None else int(kw["kv_len"][b]), kw.get("causal", False),
                               0 if kw.get("prefix") is None else int(kw["prefix"][b]), at("q_doc", b), at("k_doc", b))
                     for b in range(B_)])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["all", "causal", "lengths", "documents"])
@pytest.mark.parametrize("shape", SHAPES)
def test_odd_values_reach_those_who_see_them(shape, mode, kind):
    B_, Sq, Skv, Hq, Hkv, D, parts = shape
    assert (B.attention_workspace_bytes(*shape[:6]) > 0) == parts
    rng = np.random.default_rng(3)
    kw = _arguments(shape, mode)
    (q, qv), (k, kv), (v, vv) = _make(*shape[:6], kind, 5)
    dirty, kinds = v.clone(), np.zeros((B_, Skv, Hkv, D), int)
    places = sorted({0, 1, 31, 32, 63, 64, Skv // 2, Skv - 2, Skv - 1} | set(rng.integers(0, Skv, 6).tolist()))
    for n, j in enumerate(p for p in places if p < Skv):
        b, h, d, x = int(rng.integers(B_)), int(rng.integers(Hkv)), int(rng.integers(D)), int(rng.integers(3))
        dirty[b, j, h, d], kinds[b, j, h, d] = ODD[x], x + 1
        if n % 5 == 4:                              # a whole row
            dirty[b, j, h], kinds[b, j, h] = ODD[x], x + 1
    o = values(_gpu(q, k, dirty, **kw))
    see = _visible(shape, kw).astype(np.float64)    # [B, Sq, Skv]
    reach = np.stack([np.einsum("bij,bjhd->bihd", see, (kinds == x).astype(np.float64)) > 0 for x in (1, 2, 3)])
    reach = np.repeat(reach, Hq // Hkv, axis=3)
    nan = reach[0] | (reach[1] & reach[2])
    plus, minus = reach[1] & ~nan, reach[2] & ~nan
    assert np.array_equal(np.isnan(o), nan)
    assert np.array_equal(o == np.inf, plus) and np.array_equal(o == -np.inf, minus)
    fine = ~(nan | plus | minus)
    zeros = torch.where(torch.from_numpy(kinds > 0).cuda(), torch.zeros_like(v), v)
    clean = values(_gpu(q, k, zeros, **kw))
    assert np.array_equal(np.where(fine, o, 0.0), np.where(fine, clean, 0.0))
    if Sq * Skv * Hq <= 4e6:
        want, mean, weight, seen = O.attention(qv, kv, values(zeros), scale=D ** -0.5, **kw)
        bound = _bound(want, mean, weight, seen, D, kind, np.abs(vv).max())
        assert_within(clean, want, bound, f"{mode} {shape}")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_hidden_values_change_no_bit(shape, kind):
    """Keys of a document that no query is of, and keys past the length, hold NaN and infinities."""
    B_, Sq, Skv, Hq, Hkv, D, _ = shape
    (q, _), (k, _), (v, _) = _make(*shape[:6], kind, 6)
    n = np.full(B_, Skv - 5)
    k_doc, q_doc = np.zeros((B_, Skv), np.int32), np.zeros((B_, Sq), np.int32)
    k_doc[:, 7:11] = 1
    k_doc[:, Skv // 2:Skv // 2 + 40:3] = 2
    kw = dict(kv_len=n, k_doc=k_doc, q_doc=q_doc, causal=True)
    clean = _gpu(q, k, v, **kw)
    hidden = torch.from_numpy(k_doc != 0).cuda()
    hidden[:, Skv - 5:] = True
    for bad in ODD:
        dk, dv = k.clone(), v.clone()
        dk[hidden], dv[hidden] = bad, bad
        assert torch.equal(_gpu(q, dk, dv, **kw), clean), bad


@pytest.mark.parametrize("shape", SHAPES)
def test_odd_queries_and_keys_make_rows_of_nan(shape):
    B_, Sq, Skv, Hq, Hkv, D, _ = shape
    (q, _), (k, _), (v, _) = _make(*shape[:6], "bf16", 7)
    clean = values(_gpu(q, k, v, causal=True))
    dq = q.clone()
    dq[0, Sq // 2, Hq - 1, 3] = float("nan")
    o = values(_gpu(dq, k, v, causal=True))
    assert np.isnan(o[0, Sq // 2, Hq - 1]).all()
    o[0, Sq // 2, Hq - 1] = clean[0, Sq // 2, Hq - 1]
    assert np.array_equal(o, clean)
    dk = k.clone()
    at = Skv - 1 - (Sq - 1) // 2                    # seen by the queries from here on
    dk[0, at, 0, D - 1] = float("nan")
    o = values(_gpu(q, dk, v, causal=True))
    first, G = at - (Skv - Sq), Hq // Hkv
    assert np.isnan(o[0, first:, :G]).all()
    o[0, first:, :G] = clean[0, first:, :G]
    assert np.array_equal(o, clean)


@pytest.mark.parametrize("Sq,H", [(1, 2), (200, 160)])
def test_large_finite_values(Sq, H):
    """Values whose weighted sum overflows while the running maximum lags behind, but not with weights up to 1."""
    D, Skv = 64, 200
    rise = torch.linspace(0, 5.4, Skv, device="cuda")                # up to 2^7.8: no rescaling on the way
    k = (rise[None, :, None, None] * torch.ones((1, Skv, H // 2, D), device="cuda")).bfloat16()
    q = torch.ones((1, Sq, H, D), dtype=torch.bfloat16, device="cuda")
    v = torch.full((1, Skv, H // 2, D), 1e36, dtype=torch.bfloat16, device="cuda")
    o = values(_gpu(q, k, v, scale=1.0 / D))
    want = float(v[0, 0, 0, 0])
    assert np.all(np.abs(o - want) <= 2 * 2.0**-8 * want)


def test_one_odd_value_costs_a_second_pass_only():
    """A NaN that all rows see: another pass over the tiles, not one over the keys row by row (which would take
    some hundred times as long).  Ten times covers the look through each tile; 200 a mark for every value."""
    (q, _), (k, _), (v, _) = _make(1, 2048, 2048, 8, 8, 128, "bf16", 8)
    ws, o = B.attention_workspace(q, k), torch.empty_like(q)
    one, every = v.clone(), torch.full_like(v, float("nan"))
    one[0, 1000, :, 5] = float("nan")

    def time(value):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t = []
        for _ in range(6):
            e[0].record()
            B.attention(q, k, value, o, ws)
            e[1].record()
            torch.cuda.synchronize()
            t.append(e[0].elapsed_time(e[1]))
        return float(np.median(t[1:]))

    plain, a, b = time(v), time(one), time(every)
    print(f"{1e3 * plain:.1f} us, one NaN {1e3 * a:.1f}, all {1e3 * b:.1f}")
    assert a <= 10 * plain and b <= 200 * plain
    assert torch.isnan(o).all()
