"""Rotary positions against the 64-bit oracle.

Bound: the angle is off by at most 2^-24 of a turn from its fraction's
rounding and as much from hi + lo and the position's product (under 2^-20
radians), sine and cosine by 2^-22, the products by 2^-23: under 2^-19 of
|a| + |b|, and half an ulp of the store."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import assert_within, device, half_ulp, values

pytestmark = pytest.mark.gpu


def _check(y, x, pos, dims, theta, shared, inter, kind, what):
    want, mag = O.rope(x, O.rope_angles(pos, dims, theta, shared), inter)
    assert_within(values(y), want, np.where(mag > 0, mag * 2.0**-19 + half_ulp(np.abs(want) + mag * 2.0**-19, kind), 0),
                  what)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("M,H,H2,D,dims,shared,top", [
    (1, 1, 0, 16, [16], False, 10), (3, 24, 24, 128, [16, 56, 56], False, 128), (17, 32, 8, 128, [44, 42, 42], True, 4096),
    (5, 3, 1, 64, [16, 24, 24], False, 100), (7, 2, 2, 80, [32], False, 1 << 20), (2, 5, 3, 24, [16], False, 3),
    (1100, 6, 2, 64, [32, 0, 32], True, 70000), (4, 300, 1, 72, [64], False, (1 << 24) - 1), (9, 1, 1, 512, [512], False, 9000),
    (6, 7, 0, 256, [0, 128, 16, 16, 16, 16, 16, 48], False, 500), (2100, 24, 24, 128, [16, 56, 56], False, 64)])
def test_against_oracle(kind, inter, M, H, H2, D, dims, shared, top):
    rng = np.random.default_rng(M + D)
    plan = B.RopePlan(dims, 10000.0, shared, inter)
    pos = rng.integers(-top, top + 1, (M, len(dims))).astype(np.int32)
    pd = torch.from_numpy(pos).cuda()
    # queries, keys and values side by side, as a projection writes them
    qkv, v = device(rng.standard_normal((M, H + 2 * H2, D)), kind)
    y = torch.full((M, H, D), float("nan"), dtype=qkv.dtype, device="cuda")
    y2 = torch.full((M, H2, D), float("nan"), dtype=qkv.dtype, device="cuda") if H2 else None
    B.rope(plan, pd, qkv[:, :H], y, qkv[:, H:H + H2] if H2 else None, y2)
    _check(y, v[:, :H], pos, dims, 10000.0, shared, inter, kind, "queries")
    if H2:
        _check(y2, v[:, H:H + H2], pos, dims, 10000.0, shared, inter, kind, "keys")
    assert np.array_equal(values(qkv), v)
    # in place: the same bits, and nothing else touched
    B.rope(plan, pd, qkv[:, :H], qkv[:, :H], qkv[:, H:H + H2] if H2 else None, qkv[:, H:H + H2] if H2 else None)
    assert torch.equal(qkv[:, :H], y) and (not H2 or torch.equal(qkv[:, H:H + H2], y2))
    assert np.array_equal(values(qkv[:, H + H2:]), v[:, H + H2:])


def test_position_zero_is_the_identity_and_turns_add_up():
    plan = B.RopePlan([16, 24, 24], 10000.0)
    x, xv = device(np.random.default_rng(1).standard_normal((6, 4, 64)), "fp16")
    zero = torch.zeros((6, 3), dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    B.rope(plan, zero, x, y)
    assert torch.equal(x, y)
    # forth and back again
    pos = torch.randint(-500, 500, (6, 3), dtype=torch.int32, device="cuda")
    z = torch.empty_like(x)
    B.rope(plan, pos, x, y)
    B.rope(plan, -pos, y, z)
    assert np.abs(values(z) - xv).max() <= 4 * 2.0**-11 * np.abs(xv).max()


def test_heads_apart_and_tokens_inside():
    """A layout with heads outermost, as a cache keeps them."""
    rng = np.random.default_rng(2)
    plan = B.RopePlan([16, 24, 24], 10000.0, interleaved=False)
    x, xv = device(rng.standard_normal((11, 5, 64)), "bf16")
    pos = rng.integers(0, 99, (11, 3)).astype(np.int32)
    cache = torch.zeros((5, 40, 72), dtype=torch.bfloat16, device="cuda")
    view = cache[:, 20:31, 8:].transpose(0, 1)
    B.rope(plan, torch.from_numpy(pos).cuda(), x, view)
    _check(view, xv, pos, [16, 24, 24], 10000.0, False, False, "bf16", "cache")
    cache[:, 20:31, 8:] = 0
    assert not cache.any()


def test_infinity_and_nan_stay_in_their_pair():
    plan = B.RopePlan([32], 10000.0)
    x, _ = device(np.ones((1, 2, 32)), "bf16")
    x[0, 1, 6] = float("nan")
    x[0, 0, 30] = float("inf")
    y = torch.empty_like(x)
    B.rope(plan, torch.full((1, 1), 3, dtype=torch.int32, device="cuda"), x, y)
    bad = ~np.isfinite(values(y))
    assert set(zip(*np.nonzero(bad))) == {(0, 1, 6), (0, 1, 7), (0, 0, 30), (0, 0, 31)}


def test_stream_and_refusals():
    plan = B.RopePlan([16], 10000.0)
    x, xv = device(np.random.default_rng(3).standard_normal((8, 2, 16)), "bf16")
    pos = torch.arange(8, dtype=torch.int32, device="cuda")[:, None].contiguous()
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.rope(plan, pos, x, y, stream=side)
    side.synchronize()
    _check(y, xv, pos.cpu().numpy(), [16], 10000.0, False, True, "bf16", "stream")
    wide = torch.empty((8, 2, 20), dtype=torch.bfloat16, device="cuda")[..., :16]     # strides of 20
    for a in [(pos.long(), x, y), (pos[:4], x, y), (pos, x.float(), y), (pos, x, y.half()), (pos, x[:, :, :8], y[:, :, :8]),
              (pos, x, y[:, :1]), (pos, x.cpu(), y), (pos, x, y, x), (pos, x, y, x[:4], y[:4]), (pos, wide, y), (pos, x[0], y[0]),
              (pos.cpu(), x, y), (pos, x[:, :, ::2], y)]:
        with pytest.raises(B.SvdqError):
            B.rope(plan, *a)
