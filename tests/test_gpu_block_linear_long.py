"""The FP8 linear at its largest K in each arrangement, and groups of waves
with uneven numbers of steps.  Bounds as in tests/test_gpu_block_linear.py."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import assert_within, half_ulp, values
from tests.test_gpu_block_linear import _check, _operands, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [
    (33, 65536, 4112), (50, 1152, 4160), (64, 1408, 4160),   # 64 x 32, four groups: 512, 9 and 11 steps
    (20, 65536, 2064), (20, 1408, 2064)])                    # 32 x 32, eight groups: 512 and 11 steps
def test_small_tiles(M, K, N):
    xq, xs, wq, ws = _operands(M, K, N, M + K + N)
    y, mag = O.fp8_linear(xq, xs, wq, ws)
    Y = _run(xq, xs, wq, ws, "bf16")
    _check(Y, y, mag, K, "bf16", f"{M}x{K}x{N}")
    assert torch.equal(Y, _run(xq, xs, wq, ws, "bf16")), "two runs differ"


def test_blocks_sharing_the_largest_k():
    M, K, N = 129, 65536, 1552
    xq, xs, wq, ws = _operands(M, K, N, 5, "normal")
    assert B.fp8_linear_workspace_bytes(M, K, N) > 0
    y, mag = O.fp8_linear(xq, xs, wq, ws)
    _check(_run(xq, xs, wq, ws, "bf16"), y, mag, K, "bf16", "shared")


@pytest.mark.parametrize("M,N", [(200, 2512),      # 64 x 64, four groups
                                 (4100, 2064)])    # 128 x 128
def test_tiles_without_sharing_at_the_largest_k(M, N):
    """svdq_fp8_linear itself, which has no workspace; sampled rows."""
    K = 65536
    rng = np.random.default_rng(6)
    xq, wq = (rng.integers(0, 120, s, dtype=np.uint8) for s in ((M, K), (N, K)))
    xq[:, ::3] |= 0x80
    xs = np.exp(rng.uniform(-6, -2, (M, K // 128))).astype(np.float32)
    ws = np.exp(rng.uniform(-6, -2, (-(-N // 128), K // 128))).astype(np.float32)
    d = [torch.from_numpy(a).cuda() for a in (xq, xs, wq, ws)]
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert B.lib().svdq_fp8_linear(*(t.data_ptr() for t in d), None, M, K, N, 0, Y.data_ptr(), s) == 0
    torch.cuda.synchronize()
    assert bool(torch.isfinite(Y.float()).all())
    rows = [0, M // 2 + 1, M - 1]
    y, mag = O.fp8_linear(xq[rows], xs[rows], wq, ws)
    e = (256 + K / 128 + 8) * 2.0**-24 * mag + 2.0**-22 * np.abs(y)
    assert_within(values(Y[rows]), y, half_ulp(np.abs(y) + e, "bf16") + e, f"{M}x{K}x{N}")
