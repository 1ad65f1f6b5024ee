"""The FP8 linear against the 64-bit oracle.

Bound: a block sum adds 128 products in the matrix unit's fp32 (at most 2^-23
of the sum of magnitudes for each addition, as for truncation), the blocks are
added in fp32 with three roundings each: e = (256 + K / 128 + 8) 2^-24 sum
|x w|; the store adds half an ulp."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import DTYPES, assert_within, device, half_ulp, values

pytestmark = pytest.mark.gpu


def _operands(M, K, N, seed, codes="all"):
    rng = np.random.default_rng(seed)
    def draw(rows):
        if codes == "all":      # every finite code
            c = rng.integers(0, 254, (rows, K))
            return np.where(c >= 127, c + 1, c).astype(np.uint8)
        return O.e4m3_encode(np.clip(rng.standard_normal((rows, K)) * 100, -448, 448))
    xq, wq = draw(M), draw(N)
    xs = np.exp(rng.uniform(-6, 2, (M, K // 128))).astype(np.float32)
    ws = np.exp(rng.uniform(-6, 2, (-(-N // 128), K // 128))).astype(np.float32)
    return xq, xs, wq, ws


def _run(xq, xs, wq, ws, kind, bias=None, stream=None):
    t = lambda a: torch.from_numpy(a).cuda()
    Y = torch.full((xq.shape[0], wq.shape[0]), float("nan"), dtype=DTYPES[kind], device="cuda")
    B.fp8_linear(t(xq), t(xs), t(wq), t(ws), Y, bias=bias, stream=stream)
    torch.cuda.synchronize()
    return Y


def _check(Y, y, mag, K, kind, what):
    e = (256 + K / 128 + 8) * 2.0**-24 * mag + 2.0**-22 * np.abs(y)
    assert_within(values(Y), y, half_ulp(np.abs(y) + e, kind) + e, what)


SHAPES = [
    (1, 128, 16), (1, 3072, 9216), (2, 256, 144), (7, 1152, 272), (15, 384, 128), (16, 384, 400), (17, 640, 112),
    (31, 2048, 4096), (33, 128, 16), (48, 896, 1040), (63, 256, 2064), (64, 512, 256), (65, 384, 384), (100, 1280, 3072),
    (127, 768, 528), (129, 128, 144), (200, 4096, 272), (255, 256, 512), (257, 640, 1296), (300, 1536, 2304),
    (511, 384, 784), (513, 256, 4112), (1000, 1024, 1040), (1025, 128, 2064), (2049, 384, 528), (4100, 256, 272)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_against_oracle(M, K, N, kind):
    xq, xs, wq, ws = _operands(M, K, N, M + 31 * K + N, "normal" if kind == "fp16" else "all")
    if kind == "fp16":
        ws *= np.float32(2.0**-12)
    bd, bv = device(np.random.default_rng(1).standard_normal(N), kind) if (M + N) % 32 == 0 else (None, None)
    y, mag = O.fp8_linear(xq, xs, wq, ws, bv)
    Y = _run(xq, xs, wq, ws, kind, bd)
    _check(Y, y, mag, K, kind, f"{kind} {M}x{K}x{N}")
    assert torch.equal(Y, _run(xq, xs, wq, ws, kind, bd)), "two runs differ"


@pytest.mark.parametrize("M,K,N", [
    (2300, 384, 2320), (1283, 1152, 4144),          # 96 x 128 tiles, ragged both ways, odd steps
    (333, 2176, 3088), (200, 1152, 2064),           # 64 x 64, waves in two and four turns
    (70, 4224, 1040), (20, 65536, 144), (40, 8320, 2048),   # 64 x 32 and 32 x 32; the largest K
    (1, 65536, 16), (1, 128, 16), (1, 640, 8192), (9, 65536, 32)])
def test_each_arrangement_at_ragged_sizes(M, K, N):
    xq, xs, wq, ws = _operands(M, K, N, M + K + N)
    bd, bv = device(np.random.default_rng(2).standard_normal(N), "bf16")
    y, mag = O.fp8_linear(xq, xs, wq, ws, bv)
    Y = _run(xq, xs, wq, ws, "bf16", bd)
    _check(Y, y, mag, K, "bf16", f"{M}x{K}x{N}")
    assert torch.equal(Y, _run(xq, xs, wq, ws, "bf16", bd)), "two runs differ"


@pytest.mark.parametrize("M,K,N", [
    (690, 1152, 2960),                              # 96 x 128 tiles, two groups
    (1010, 640, 3088),                              # 128 x 128, two groups
    (1500, 1152, 3088),                             # 96 x 128
    (2300, 640, 3088)])                             # 128 x 128
def test_large_tiles_at_ragged_sizes(M, K, N):
    xq, xs, wq, ws = _operands(M, K, N, M + K + N)
    bd, bv = device(np.random.default_rng(4).standard_normal(N), "fp16")
    ws *= np.float32(2.0**-16)
    y, mag = O.fp8_linear(xq, xs, wq, ws, bv)
    Y = _run(xq, xs, wq, ws, "fp16", bd)
    _check(Y, y, mag, K, "fp16", f"{M}x{K}x{N}")
    assert torch.equal(Y, _run(xq, xs, wq, ws, "fp16", bd)), "two runs differ"


def test_every_row_and_column_is_its_own():
    """One nonzero code in each operand: exactly one output is nonzero, for places all over a ragged shape."""
    M, K, N = 270, 512, 656
    for m, k, n in [(0, 0, 0), (269, 511, 655), (255, 127, 255), (256, 128, 256), (17, 300, 639), (128, 383, 127)]:
        xq, wq = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
        xq[m, k], wq[n, k] = 0x3C, 0xC4           # 1.5 and -3
        xs = np.arange(1, 1 + M * 4, dtype=np.float32).reshape(M, 4)
        ws = np.arange(1, 1 + 24, dtype=np.float32).reshape(6, 4)
        y = values(_run(xq, xs, wq, ws, "bf16"))
        want = -4.5 * xs[m, k // 128] * ws[n // 128, k // 128]
        assert abs(y[m, n] - want) <= half_ulp(want, "bf16")
        y[m, n] = 0
        assert not y.any(), (m, k, n)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_nan_codes_and_scales_reach_only_their_outputs(M):
    K, N = 384, 320
    xq, xs, wq, ws = _operands(M, K, N, 9)
    xq[M - 1, 200] = 0x7F
    wq[5, 3] = 0xFF
    ws[2, 1] = np.inf
    y = values(_run(xq, xs, wq, ws, "bf16"))
    fine = np.ones((M, N), bool)
    fine[M - 1], fine[:, 5], fine[:, 256:] = False, False, False
    assert np.isnan(y[M - 1]).all() and np.isnan(y[:, 5]).all() and not np.isfinite(y[:, 256:]).any()
    assert np.isfinite(y[fine]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_large_shape_on_sampled_rows(kind):
    M, K, N = 4096, 3072, 9216
    rng = np.random.default_rng(11)
    xq, xs, wq, ws = _operands(M, K, N, 12, "normal")
    ws *= np.float32(2.0**-14)
    Y = _run(xq, xs, wq, ws, kind)
    rows = np.unique(np.concatenate([rng.integers(0, M, 40), [0, 255, 256, M - 1]]))
    y, mag = O.fp8_linear(xq[rows], xs[rows], wq, ws)
    e = (256 + K / 128 + 8) * 2.0**-24 * mag + 2.0**-22 * np.abs(y)
    assert_within(values(Y[torch.from_numpy(rows).cuda()]), y, half_ulp(np.abs(y) + e, kind) + e, kind)


def test_stream_and_refusals():
    xq, xs, wq, ws = _operands(20, 256, 144, 13)
    y, mag = O.fp8_linear(xq, xs, wq, ws)
    side = torch.cuda.Stream()
    Y = _run(xq, xs, wq, ws, "bf16", stream=side)
    _check(Y, y, mag, 256, "bf16", "stream")
    t = lambda a: torch.from_numpy(a).cuda()
    good = dict(xq=t(xq), xs=t(xs), wq=t(wq), ws=t(ws), Y=Y)
    f8 = torch.float8_e4m3fn
    Y2 = torch.empty_like(Y)
    B.fp8_linear(good["xq"].view(f8), good["xs"], good["wq"].view(f8), good["ws"], Y2)
    assert torch.equal(Y, Y2)
    for change in [dict(xq=good["xq"].cpu()), dict(xq=good["xq"].to(torch.int32)), dict(wq=good["wq"][:, :128]),
                   dict(xs=good["xs"][:, :1]), dict(xs=good["xs"].double()), dict(ws=good["ws"][:1]),
                   dict(Y=Y.float()), dict(Y=Y[:, :128]), dict(Y=Y.t()), dict(bias=Y[0].float()),
                   dict(bias=Y[0, :128].contiguous()), dict(xq=good["xq"][:, ::2])]:
        a = dict(good)
        a.update(change)
        with pytest.raises(B.SvdqError):
            B.fp8_linear(**a)


SHARED = [(129, 12288, 1552), (700, 8320, 1552), (2900, 16384, 144), (333, 12416, 3088), (128, 12288, 3072)]


@pytest.mark.parametrize("M,K,N", SHARED)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_blocks_sharing_k(M, K, N, kind):
    """Uneven parts and ragged edges; a used, larger workspace and torch's own give the same bits."""
    xq, xs, wq, ws = _operands(M, K, N, M + K + N, "normal")
    ws *= np.float32(2.0**-14)
    bd, bv = device(np.random.default_rng(3).standard_normal(N), kind)
    y, mag = O.fp8_linear(xq, xs, wq, ws, bv)
    n = B.fp8_linear_workspace_bytes(M, K, N)
    assert n > 0
    Y = _run(xq, xs, wq, ws, kind, bd)
    _check(Y, y, mag, K, kind, f"{kind} {M}x{K}x{N}")
    t = lambda a: torch.from_numpy(a).cuda()
    a = dict(xq=t(xq), xs=t(xs), wq=t(wq), ws=t(ws), bias=bd)
    for w in (torch.full((n + 1024,), 255, dtype=torch.uint8, device="cuda"), None):
        Y2 = torch.full_like(Y, float("nan"))
        B.fp8_linear(Y=Y2, workspace=w, **a)
        assert torch.equal(Y, Y2)
    with pytest.raises(B.SvdqError):
        B.fp8_linear(Y=Y2, workspace=w or torch.empty(n - 16, dtype=torch.uint8, device="cuda"), **a)
    with pytest.raises(B.SvdqError):
        B.fp8_linear(Y=Y2, workspace=torch.empty(n, dtype=torch.int8, device="cuda"), **a)


def test_blocks_sharing_k_on_two_streams_and_in_a_graph():
    M, K, N = 129, 12288, 1552
    t = lambda a: torch.from_numpy(a).cuda()
    ops = [[t(a) for a in _operands(M, K, N, seed, "normal")] for seed in (1, 2)]
    want = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in ops]
    for o, y in zip(ops, want):
        B.fp8_linear(*o, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[torch.zeros_like(want[0]) for _ in range(4)] for _ in ops]
    torch.cuda.synchronize()
    for i in range(4):
        for o, y, s in zip(ops, got, streams):
            B.fp8_linear(*o, y[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)
    g, out = torch.cuda.CUDAGraph(), [torch.zeros_like(w) for w in want]
    with torch.cuda.graph(g):
        for o, y in zip(ops, out):
            B.fp8_linear(*o, y)
    for _ in range(3):
        for y in out:
            y.zero_()
        g.replay()
        B.fp8_linear(*ops[0], got[0][0])
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(out, want))
