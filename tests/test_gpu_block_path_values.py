"""A first token through examples/attention_block.py, step by step: the
residual sum, the codes and the V columns of the projection that the cache
holds, against the 64-bit oracle on the device's own codes."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import assert_within, half_ulp, values
from tests.test_gpu_block_path import _module

pytestmark = pytest.mark.gpu


def test_what_the_first_token_leaves():
    width, D = 256, 64
    b = _module().AttentionBlock(width, 2, 1, D, (16, 24, 24), 4, rank=16)
    x, r = (torch.randn((1, width), device="cuda").bfloat16() for _ in range(2))
    h, o, _ = b(x, torch.tensor([[5, 6, 7]], dtype=torch.int32, device="cuda"), r)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    q, s = torch.empty((1, width), dtype=torch.uint8, device="cuda"), torch.empty((1, 2), device="cuda")
    B.add_rmsnorm_quantize(x, b.norm, 1e-6, q, s, residual=r)
    _, y, sc = O.add_rmsnorm(values(x), values(b.norm), 1e-6, values(r))
    assert_within(s.cpu().numpy(), sc, sc * 2.0**-18, "scales")
    codes = q.cpu().numpy()
    back = O.fp8_dequant(codes, s.cpu().numpy(), 1)
    assert_within(back, y, np.maximum(np.abs(y) * 2.0**-4, np.repeat(sc, 128, 1) * 2.0**-10) + 2.0**-17 * np.abs(y), "codes")
    want, mag = O.fp8_linear(codes, s.cpu().numpy(), b.wqkv.view(torch.uint8).cpu().numpy(), b.sqkv.cpu().numpy(),
                             values(b.bqkv))
    v, m = want[0, 3 * D:], mag[0, 3 * D:]
    e = (256 + width / 128 + 8) * 2.0**-24 * m + 2.0**-22 * np.abs(v)
    bound = half_ulp(np.abs(v) + e, "bf16") + e
    assert_within(values(b.v[0, 0, 0]), v, bound, "V")
    assert np.array_equal(values(o).reshape(2, D), np.stack([values(b.v[0, 0, 0])] * 2))
    assert not b.k[0, 1:].any() and not b.v[0, 1:].any()
