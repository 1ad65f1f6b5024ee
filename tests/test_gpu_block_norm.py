"""Residual sum + RMS norm + FP8 codes against the 64-bit oracle.

Bounds.  h is the fp32 sum rounded to 16 bits: equal bits.  The sum of
squares has at most 64 sequential fp32 additions and 22 levels of exchange on
positive terms, halved by the root, plus five roundings up to the scale: under
64 units of 2^-24, so 2^-18 relative on y and s.  A code stands for a value
within half a spacing of E4M3 (2^-4 of y, or 2^-10 s among subnormals) of y,
widened by that 2^-18 twice (y and s)."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import DTYPES, assert_within, device, values

pytestmark = pytest.mark.gpu


def _call(x, w, eps, r=None, h=None, stream=None):
    M, K = x.shape
    q = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M, -(-K // 128)), -7.0, dtype=torch.float32, device="cuda")
    B.add_rmsnorm_quantize(x, w, eps, q, s, residual=r, h=h, stream=stream)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def _check(q, s, xv, wv, eps, rv, what):
    _, y, sc = O.add_rmsnorm(xv, wv, eps, rv)
    assert_within(s, sc, sc * 2.0**-18, what + " scales")
    back = O.fp8_dequant(q, s, 1)
    sb = np.repeat(sc, 128, axis=1)[:, :y.shape[1]]
    assert_within(back, y, np.maximum(np.abs(y) * 2.0**-4, sb * 2.0**-10) + 2.0**-17 * np.abs(y), what + " codes")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", [
    (1, 8), (3, 16), (5, 120), (4, 128), (7, 136), (2, 248), (9, 512), (1, 520), (33, 1000), (6, 3072), (1, 3072),
    (5, 4096), (3, 4104), (2, 8192), (1, 12288), (3, 20000), (2, 65536), (1, 65528), (1031, 264)])
def test_against_oracle(kind, residual, M, K):
    rng = np.random.default_rng(M * 70001 + K)
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 30.0, 1.0)
    xd, xv = device(x, kind)
    wd, wv = device(1 + 0.2 * rng.standard_normal(K), kind)
    rd, rv = device(3 * rng.standard_normal((M, K)), kind) if residual else (None, None)
    h = torch.empty_like(xd)
    q, s = _call(xd, wd, 1e-6, rd, h)
    h32 = xd.float() if rd is None else xd.float() + rd.float()
    assert torch.equal(h, h32.to(DTYPES[kind])), "h"
    _check(q, s, xv, wv, 1e-6, rv, f"{kind} {M}x{K}")
    q2, s2 = _call(xd, wd, 1e-6, rd)           # h not asked for: the same codes
    assert np.array_equal(q, q2) and np.array_equal(s, s2)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("K", [384, 6144])
def test_strided_rows_and_in_place(kind, target, K):
    rng = np.random.default_rng(K)
    M = 37
    big, _ = device(rng.standard_normal((M, K + 40)), kind)
    other, _ = device(rng.standard_normal((M, 2 * K)), kind)
    x, r = big[:, 16:16 + K], other[:, K:]
    xv, rv = values(x), values(r)
    wd, wv = device(1 + 0.2 * rng.standard_normal(K), kind)
    keep_big, keep_other = big.clone(), other.clone()
    h32 = (x.float() + r.float()).to(DTYPES[kind])
    h = x if target == "x" else r
    q, s = _call(x, wd, 1e-5, r, h)
    assert torch.equal(h, h32)
    _check(q, s, xv, wv, 1e-5, rv, f"in place {target}")
    # nothing outside the rows' own columns was written
    big[:, 16:16 + K] = 0
    keep_big[:, 16:16 + K] = 0
    other[:, K:] = 0
    keep_other[:, K:] = 0
    assert torch.equal(big, keep_big) and torch.equal(other, keep_other)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_zero_rows_and_blocks(kind):
    M, K = 4, 384
    x = np.random.default_rng(5).standard_normal((M, K))
    x[0] = 0.0                        # a row of zeros
    x[1, 128:256] = 0.0               # a block of zeros
    x[2, 1:] = 0.0                    # one value alone
    xd, xv = device(x, kind)
    wd, wv = device(np.ones(K), kind)
    q, s = _call(xd, wd, 1e-6)
    assert not q[0].any() and not s[0].any() and not q[1, 128:256].any() and s[1, 1] == 0
    _check(q, s, xv, wv, 1e-6, None, "zeros")
    q, s = _call(xd, wd, 0.0)         # eps 0 and a zero row: 0 * infinity
    assert np.isnan(s[0]).all() and np.all(q[0] & 0x7F == 0x7F)
    _check(q[1:], s[1:], xv[1:], wv, 0.0, None, "eps 0")


def test_scale_below_the_normal_range_gives_zero_codes():
    xd, _ = device(np.ones((1, 256)), "bf16")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    w[:128] = 1e-38                   # |y| / 448 is below 2^-126
    w[128:] = 1e-30
    q, s = _call(xd, w, 0.0)
    assert s[0, 0] == 0 and not q[0, :128].any()
    assert abs(s[0, 1] * 448 / float(w[128]) - 1) < 1e-5 and np.all(q[0, 128:] == 0x7E)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_nan_and_infinity(kind):
    M, K = 3, 512
    x = np.random.default_rng(6).standard_normal((M, K)).astype(np.float32)
    x[0, 130] = np.nan
    x[1, 300] = np.inf
    xd, xv = device(x, kind)
    wd, wv = device(np.ones(K), kind)
    q, s = _call(xd, wd, 1e-6)
    nan = (q & 0x7F) == 0x7F
    assert nan[0].all() and np.isnan(s[0]).all()                    # the row's norm is NaN
    assert nan[1, 300] and nan[1].sum() == 1 and not (q[1] & 0x7F)[~nan[1]].any()
    assert np.isnan(s[1, 2]) and not s[1, [0, 1, 3]].any()          # an infinite norm: the rest of the row is 0
    _check(q[2:], s[2:], xv[2:], wv, 1e-6, None, "the row beside them")


def test_nan_in_the_weight_stays_in_its_block():
    xd, _ = device(np.random.default_rng(7).standard_normal((2, 256)), "bf16")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    w[200] = float("nan")
    q, s = _call(xd, w, 1e-6)
    nan = (q & 0x7F) == 0x7F
    assert np.isnan(s[:, 1]).all() and nan[:, 200].all() and nan.sum() == 2 and np.isfinite(s[:, 0]).all()
    assert not (q[:, 128:] & 0x7F)[~nan[:, 128:]].any()


def test_other_stream_and_refusals():
    xd, xv = device(np.random.default_rng(8).standard_normal((64, 1024)), "bf16")
    wd, wv = device(np.ones(1024), "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = _call(xd, wd, 1e-6, stream=side)
    _check(q, s, xv, wv, 1e-6, None, "stream")
    q8 = torch.empty((64, 1024), dtype=torch.float8_e4m3fn, device="cuda")
    s8 = torch.empty((64, 8), dtype=torch.float32, device="cuda")
    B.add_rmsnorm_quantize(xd, wd, 1e-6, q8, s8)
    assert np.array_equal(q8.view(torch.uint8).cpu().numpy(), q)
    bad = [dict(x=xd.float()), dict(x=xd.cpu()), dict(x=xd[:, ::2]), dict(weight=wd[:512]), dict(weight=wd.half()),
           dict(q=q8[:, :512]), dict(q=q8.to(torch.float32)), dict(s=s8[:, :4]), dict(s=s8.double()),
           dict(residual=xd[:32]), dict(residual=xd.half()), dict(h=xd.float()), dict(x=xd[0])]
    for change in bad:
        a = dict(x=xd, weight=wd, eps=1e-6, q=q8, s=s8)
        a.update(change)
        with pytest.raises(B.SvdqError):
            B.add_rmsnorm_quantize(**a)
