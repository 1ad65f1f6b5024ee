"""The score cap over its whole accepted range, against the 64-bit oracle.

Bound: that of tests/test_gpu_block_attention.py with the magnitudes of the
score without its cap: cap tanh(score / cap) has slope at most 1 and is never
larger than the score, and a tanh good to a few units of 2^-24 relative is
covered by the allowance of (2 D + 16) units on 4 |score|.  Nothing of the
cap's own size enters, so a large cap has to be as exact as none."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import assert_within, device, values
from tests.test_gpu_block_attention import _bound, _gpu, _make

pytestmark = pytest.mark.gpu

CAPS = [1e-42, 1e-20, 5.0, 50.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e8, 1e30, 3e38]
# one token, few rows with shared heads, blocks of 128 rows, and those with parts
SHAPES = [(2, 1, 2000, 4, 2, 64), (1, 5, 700, 6, 2, 128), (6, 129, 200, 16, 8, 104), (1, 700, 2100, 4, 4, 64)]


def _check(o, qv, kv, vv, kind, what, **kw):
    want, mean, _, seen = O.attention(qv, kv, vv, **kw)
    free = dict(kw, softcap=0.0)
    weight = O.attention(qv, kv, vv, **free)[2]
    assert_within(values(o), want, _bound(want, mean, weight, seen, qv.shape[-1], kind, np.abs(vv).max()), what)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_caps_of_every_size(kind, shape):
    (q, qv), (k, kv), (v, vv) = _make(*shape, kind, 17)
    q[:, 0] = 0                                     # a query of zeros: all its scores are 0 under any cap
    qv[:, 0] = 0
    for cap in CAPS:
        kw = dict(scale=shape[-1] ** -0.5, softcap=cap, causal=True)
        _check(_gpu(q, k, v, **kw), qv, kv, vv, kind, f"cap {cap}", **dict(kw, softcap=float(np.float32(cap))))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("Sq,H", [(1, 2), (200, 2), (200, 160)])
def test_scores_around_the_cap(kind, Sq, H):
    """Scores far below, at and far above the cap in one row, of both signs and under both signs of the scale."""
    D, Skv = 64, 300
    steps = np.concatenate([[0.0], np.geomspace(1e-6, 4.0, (Skv - 1) // 2), -np.geomspace(1e-6, 4.0, Skv - 1 - (Skv - 1) // 2)])
    k, kv = device(steps[None, :, None, None] * np.ones((1, Skv, H // 2, D)), kind)
    q, qv = device(np.ones((1, Sq, H, D)), kind)
    v, vv = device(np.random.default_rng(18).standard_normal((1, Skv, H // 2, D)), kind)
    for cap in (3.0, 0.5):
        for scale in (cap / D, -cap / D):           # |score| from nothing to four times the cap
            kw = dict(scale=scale, softcap=cap)
            _check(_gpu(q, k, v, **kw), qv, kv, vv, kind, f"cap {cap} scale {scale}", **kw)


def test_a_large_cap_is_as_good_as_none():
    (q, _), (k, _), (v, _) = _make(2, 70, 900, 8, 2, 128, "bf16", 19)
    free = values(_gpu(q, k, v))
    far = values(_gpu(q, k, v, softcap=1e7))        # scores of about 10: tanh(x) = x within 1e-12
    assert np.abs(far - free).max() <= 2 * 2.0**-8 * np.abs(free).max()


@pytest.mark.parametrize("Sq,H", [(1, 2), (200, 160)])
@pytest.mark.parametrize("cap", [0.0, 1.0, 1e6])
def test_the_largest_scales_leave_scores_of_zero(Sq, H, cap):
    """Times log2 e they leave fp32; a query of zeros still weighs its keys alike."""
    D, Skv = 64, 150
    (_, _), (k, _), (v, vv) = _make(1, Sq, Skv, H, H // 2, D, "bf16", 20)
    q = torch.zeros((1, Sq, H, D), dtype=torch.bfloat16, device="cuda")
    want = np.repeat(vv.mean(1), 2, axis=1)[:, None]
    for scale in (3e38, -3e38, 1e-45):
        o = values(_gpu(q, k, v, scale=scale, softcap=cap))
        assert np.abs(o - want).max() <= 2.0**-7 * np.abs(vv).mean(1).max(), scale
