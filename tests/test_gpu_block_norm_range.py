"""The norm over the whole range of bf16.

Bounds as in tests/test_gpu_block_norm.py: scaling a row by a power of two is
exact, so rows whose squares leave fp32's range are held to the same."""
import numpy as np
import pytest

from tests.block_util import device
from tests.test_gpu_block_norm import _call, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(1, 3072), (4, 8), (3, 65536), (700, 2048), (600, 20000)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_rows_of_every_magnitude(M, K, eps):
    rng = np.random.default_rng(M + K)
    size = np.exp2(rng.integers(-126, 121, (M, 1)).astype(np.float64))
    size[0] = 2.0**110                              # squares above fp32
    size[-1] = 2.0**-75 if M > 1 else size[-1]      # and below
    w, wv = device(1 + 0.2 * rng.standard_normal(K), "bf16")
    x, xv = device(np.clip(rng.standard_normal((M, K)) * size, -3e38, 3e38), "bf16")
    q, s = _call(x, w, eps)
    # where eps decides, y may be below the scales' range: those blocks are zero (and the oracle's y with them)
    y = xv / np.sqrt(np.mean(xv * xv, axis=1, keepdims=True) + eps) * wv
    rows = np.abs(y).max(1) > 1e-30
    assert rows[0] and rows.any()
    _check(q[rows], s[rows], xv[rows], wv, eps, None, f"{M}x{K} eps {eps}")


def test_a_large_value_in_a_row_of_small_ones():
    x = np.full((2, 512), 2.0**-100)
    x[0, 77] = 2.0**100
    x[1, 77] = 2.0**-60
    xd, xv = device(x, "bf16")
    wd, wv = device(np.ones(512), "bf16")
    q, s = _call(xd, wd, 0.0)
    assert q[0, 77] == 0x7E and abs(s[0, 0] * 448 - 512 ** 0.5) <= 2.0**-17 * 512 ** 0.5
    assert q[1, 77] == 0x7E and abs(s[1, 0] * 448 - 512 ** 0.5) <= 2.0**-17 * 512 ** 0.5
