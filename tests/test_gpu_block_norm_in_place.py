"""The norm with h in the place of x or of the residual."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from tests.test_gpu_block_norm import _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("M,K", [(1, 512), (5, 8192), (3, 65536), (600, 2048), (600, 8192), (513, 20000), (520, 65536)])
def test_in_place_in_every_arrangement(M, K, target):
    """One to eight chunks a lane, rows of one wave and of sixteen."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x, r = (torch.randn((M, K), generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    h = torch.empty_like(x)
    q, s = _call(x, w, 1e-6, r, h)
    xi, ri = x.clone(), r.clone()
    hi = xi if target == "x" else ri
    qi, si = _call(xi, w, 1e-6, ri, hi)
    assert np.array_equal(q, qi) and np.array_equal(s, si) and torch.equal(h, hi)
    assert torch.equal(*((ri, r) if target == "x" else (xi, x)))


def test_in_place_with_another_stride_is_refused():
    a = torch.randn((8, 512), device="cuda").bfloat16()
    x, h = a[:4, :256], a.view(16, 256)[:4]         # the same first row, other rows after it
    q, s = torch.empty((4, 256), dtype=torch.uint8, device="cuda"), torch.empty((4, 2), device="cuda")
    w, keep = torch.ones(256, dtype=torch.bfloat16, device="cuda"), a.clone()
    for kw in (dict(x=x), dict(x=torch.zeros_like(x), residual=x)):
        with pytest.raises(B.SvdqError) as e:
            B.add_rmsnorm_quantize(weight=w, eps=1e-6, q=q, s=s, h=h, **kw)
        assert e.value.status == 1
    assert torch.equal(a, keep)
    B.add_rmsnorm_quantize(x[:1], w, 1e-6, q[:1], s[:1], h=h[:1])     # a single row has no stride
