"""The block operators run together as examples/attention_block.py does.

A prompt at once and the same tokens in pieces (a shorter prompt, a chunk, one
token at a time) take different kernels for the linear and for attention; the
attention outputs agree to the roundings on the way: Q, K, V may differ by one
bf16 rounding (2^-8 of a value) and the weights by another, so 4 x 2^-8 of
the outputs' norm covers both.  Every output projection is checked against the
quantized linear's own oracle on the attention output the device produced, to the
method's 5e-3."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from oracle import forward as F
from oracle import prepare as P
from rank_gemm_svdq_amd import synthetic as S
from tests.block_util import values
from tests.gpu_util import rel_fro

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _module():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("heads,kv_heads,D", [(8, 2, 64), (4, 4, 128)])
def test_pieces_agree_with_the_whole(heads, kv_heads, D):
    E = _module()
    width, M = 512, 333
    axes = (16, D // 2 - 8, D // 2 - 8)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((M, width), generator=g, device="cuda").bfloat16()
    r = torch.randn((M, width), generator=g, device="cuda").bfloat16()
    at = torch.arange(M, device="cuda")
    pos = torch.stack([at // 64, at // 8 % 8, at % 8], 1).to(torch.int32)
    make = lambda: E.AttentionBlock(width, heads, kv_heads, D, axes, M + 5, rank=16)
    h, o, y = make()(x, pos, r)
    piece = make()
    parts, i = [], 0
    for n in (200, 100, 1, 1, 20, 1, 10):
        parts.append(piece(x[i:i + n], pos[i:i + n].contiguous(), r[i:i + n]))
        i += n
    assert i == M
    h2, o2, y2 = (torch.cat([p[k] for p in parts]) for k in range(3))
    assert torch.equal(h, h2)
    assert rel_fro(values(o2), values(o)) <= 4 * 2.0**-8
    # the projection on the attention output of the device
    b = make()
    po = P.prepare((S.random_bf16(0, (heads * D, width)) / (heads * D) ** 0.5).astype(np.float32),
                   np.ones(heads * D, np.float32), 0.5, 16, "mxfp4")
    for oo, yy in ((o, y), (o2, y2)):
        assert rel_fro(values(yy), F.forward(values(oo).astype(np.float32), po, None)["y"]) <= 5e-3
    assert b.prep["rank"] == 16


def test_first_token_sees_itself_alone():
    E = _module()
    b = E.AttentionBlock(256, 2, 1, 64, (16, 24, 24), 4, rank=16)
    x = torch.randn((1, 256), device="cuda").bfloat16()
    b(x, torch.zeros((1, 3), dtype=torch.int32, device="cuda"))
    b2 = E.AttentionBlock(256, 2, 1, 64, (16, 24, 24), 4, rank=16)
    _, o, _ = b2(x, torch.tensor([[5, 6, 7]], dtype=torch.int32, device="cuda"))
    v = values(b2.v[0, 0, 0])
    assert np.array_equal(values(o).reshape(2, 64), np.stack([v, v]))     # one key: its value, whatever the angle
    h, y, s = O.add_rmsnorm(values(x), values(b2.norm), 1e-6)
    assert h.shape == (1, 256) and np.isfinite(y).all()
