"""The gated residual norms against the 64-bit oracle.

Bound.  u = 2^-24.  A sum over a row has at most 32 sequential additions, 10
levels of exchange and one more step: 64 u of the sum of its magnitudes.  With e an
element's error so far, a norm of either kind makes it
  layer: e + 64 u mean |x| + mean e + u |d| for the deviation d (RMS: d = x), then
  relative 2^-18 + sum |d| e / sum (d^2 + eps) for the root (64 positive additions halved,
  five roundings), on the result;
every product or sum after it adds u of its result.  The store adds half an ulp; a code
stands for a value within half a spacing of E4M3 (2^-4 of y, or 2^-10 s among
subnormals) of y, widened by what y and its block's largest are off."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from oracle import serving as S
from tests.block_util import DTYPES, assert_within, device, half_ulp, values
from tests.serving_util import ints

pytestmark = pytest.mark.gpu
U = 2.0**-24


def _norm_error(x, e, kind, eps):
    """Error of the norm of x whose elements are off by e."""
    if kind == "none":
        return e
    mean = lambda a: a.mean(1, keepdims=True)
    d = x
    if kind == "layer":
        d = x - mean(x)
        e = e + 64 * U * mean(np.abs(x)) + mean(e) + U * np.abs(d)
    var = mean(d * d) + eps
    with np.errstate(all="ignore"):
        return e / np.sqrt(var) + np.abs(d) / np.sqrt(var) * (2.0**-18 + mean(np.abs(d) * e) / var + mean(e * e) / var)


def _errors(x, eps, residual=None, residual_scale=1.0, post="none", post_weight=None, gate=None, pre="rms", weight=None,
            scale=None, shift=None, entry=None):
    """Bounds of h and y before their stores."""
    b, e = S.norm(x, post, eps), _norm_error(x, np.zeros_like(x), post, eps)
    for f in (post_weight, None if gate is None else gate[entry]):
        if f is not None:
            b, e = b * f, e * np.abs(f)
            e = e + U * (np.abs(b) + e)
    h = b
    if residual is not None:
        h = residual_scale * residual + b
        e = e + U * (np.abs(residual_scale * residual) + np.abs(h) + e)
    y, f = S.norm(h, pre, eps), _norm_error(h, e, pre, eps)
    for w in (weight, None if scale is None else 1.0 + scale[entry]):
        if w is not None:
            y, f = y * w, f * np.abs(w)
            f = f + 2 * U * (np.abs(y) + f)
    if shift is not None:
        y = y + shift[entry]
        f = f + U * (np.abs(y) + f)
    return e, f


def _run(x, kind, outputs="hyq", stream=None, **kw):
    M, K = x.shape
    out = {}
    if "h" in outputs:
        out["h"] = torch.full((M, K), float("nan"), dtype=x.dtype, device="cuda")
    if "y" in outputs:
        out["y"] = torch.full((M, K), float("nan"), dtype=x.dtype, device="cuda")
    if "q" in outputs:
        out["q"] = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
        out["s"] = torch.full((M, -(-K // 128)), -7.0, device="cuda")
    B.gated_norm(x, stream=stream, **out, **kw)
    torch.cuda.synchronize()
    return out


def _check(out, xv, kind, what, eps=1e-6, **kw):
    h, y = S.gated_norm(xv, eps=eps, **kw)
    eh, ey = _errors(xv, eps, **kw)
    if "h" in out:
        assert_within(values(out["h"]), h, eh + half_ulp(np.abs(h) + eh, kind), what + " h")
    if "y" in out:
        assert_within(values(out["y"]), y, ey + half_ulp(np.abs(y) + ey, kind), what + " y")
    if "q" in out:
        blocks = O.blocks(y.shape[1])
        top = np.stack([np.abs(y[:, b]).max(1) for b in blocks], 1)
        off = np.stack([ey[:, b].max(1) for b in blocks], 1)
        assert_within(values(out["s"]), top / 448, (off + 4 * U * top) / 448, what + " scales")
        back = O.fp8_dequant(out["q"].cpu().numpy(), values(out["s"]), 1)
        wide = lambda a: np.repeat(a, 128, axis=1)[:, :y.shape[1]]
        bound = np.maximum(np.abs(y) * 2.0**-4, wide(top / 448) * 2.0**-10) + 2 * ey + 2 * wide(off) + 2.0**-17 * np.abs(y)
        assert_within(back, y, bound, what + " codes")


def _case(M, K, E, kind, seed, gate=True, modulate=True, residual=True, weights=True, entry=True):
    rng = np.random.default_rng(seed)
    x, xv = device(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 10.0, 1.0), kind)
    dev, host = {}, {}

    def put(name, a):
        dev[name], host[name] = device(a, kind)

    if residual:
        put("residual", 3 * rng.standard_normal((M, K)) + 0.5)
    if weights:
        put("post_weight", 1 + 0.2 * rng.standard_normal(K))
        put("weight", 1 + 0.2 * rng.standard_normal(K))
    mod, modv = device(0.4 * rng.standard_normal((E, 3 * K)), kind)
    for i, name in enumerate(("gate", "scale", "shift")):
        if gate if name == "gate" else modulate:
            dev[name], host[name] = mod[:, i * K:(i + 1) * K], modv[:, i * K:(i + 1) * K]
    e = rng.integers(0, E, M) if entry else np.arange(M) // (M // E)
    if entry:
        dev["entry"] = ints(e)
    host["entry"] = e
    return x, xv, dev, host


SHAPES = [(1, 8, 1), (3, 16, 2), (5, 120, 5), (4, 128, 1), (7, 136, 3), (1, 512, 1), (2, 520, 2), (9, 1000, 4), (33, 2056, 7),
          (1, 4096, 1), (6, 4104, 2), (2, 8192, 2), (3, 8200, 1), (2, 16384, 2), (601, 264, 3), (530, 2048, 2), (515, 2056, 5),
          (514, 5000, 2), (513, 8192, 1), (520, 16384, 4), (513, 12296, 3)]


@pytest.mark.parametrize("M,K,E", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("none", "layer"), ("layer", "none"), ("layer", "layer")])
def test_against_oracle(M, K, E, kind, post, pre):
    x, xv, dev, host = _case(M, K, E, kind, M * 70001 + K)
    kw = dict(post=post, pre=pre, residual_scale=0.75)
    out = _run(x, kind, **dev, **kw)
    _check(out, xv, kind, f"{M}x{K} {kind} {post} {pre}", **host, **kw)
    # fewer outputs: the same bits
    for some in ("h", "y", "q", "hq"):
        for n, t in _run(x, kind, some, **dev, **kw).items():
            assert torch.equal(t, out[n]), f"{some}: {n}"


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("flags", [dict(gate=False), dict(modulate=False), dict(residual=False), dict(weights=False),
                                   dict(gate=False, modulate=False, residual=False, weights=False), dict(entry=False)])
def test_parts_left_out(kind, flags):
    for M, K, E in ((6, 384, 3), (600, 1000, 2)):
        x, xv, dev, host = _case(M, K, E, kind, 17, **flags)
        out = _run(x, kind, post="rms", pre="layer", **dev)
        _check(out, xv, kind, str(flags), post="rms", pre="layer", **host)


def test_scale_or_shift_alone_and_entries_outside_are_clamped():
    M, K, E = 7, 256, 3
    x, xv, dev, host = _case(M, K, E, "bf16", 18)
    for drop in (("scale",), ("shift",), ("gate", "scale"), ("gate", "shift")):
        d, h = ({k: v for k, v in s.items() if k not in drop} for s in (dev, host))
        _check(_run(x, "bf16", **d), xv, "bf16", str(drop), **h)
    dev["entry"], host["entry"] = ints([-5, 0, 1, 2, 3, 2**31 - 1, -2**31]), np.array([0, 0, 1, 2, 2, 2, 0])
    _check(_run(x, "bf16", **dev), xv, "bf16", "entries", **host)


@pytest.mark.parametrize("M,K", [(5, 384), (5, 6144), (600, 4096)])
@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("what", ["h", "y"])
def test_in_place_and_strided(M, K, target, what):
    x, xv, dev, host = _case(M, K, 1, "bf16", 19, entry=False)
    want = _run(x, "bf16", "hy", post="rms", **dev)
    room = torch.full((2, M, K + 24), -7.0, dtype=torch.bfloat16, device="cuda")
    room[0, :, 8:K + 8], room[1, :, 8:K + 8] = x, dev["residual"]
    xs, rs = room[0, :, 8:K + 8], room[1, :, 8:K + 8]
    other = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    place = xs if target == "x" else rs
    B.gated_norm(xs, **{what: place, "h" if what == "y" else "y": other}, post="rms", **{**dev, "residual": rs})
    assert torch.equal(place, want[what]) and torch.equal(other, want["h" if what == "y" else "y"])
    room[:, :, 8:K + 8] = -7.0
    assert bool((room == -7.0).all())


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("power", [-126, -100, -70, -40, 60, 80, 100, 118])
@pytest.mark.parametrize("M,K", [(3, 512), (2, 8200)])
def test_rows_of_any_magnitude(kind, power, M, K):
    """Norms of rows whose squares leave fp32 (bf16), before the gate and after the sum."""
    rng = np.random.default_rng(20)
    x, xv = device((rng.standard_normal((M, K)) + 0.25) * 2.0**power, "bf16")
    out = _run(x, "bf16", "yq", pre=kind, eps=0.0)
    _check({"y": out["y"], "q": out["q"], "s": out["s"]}, xv, "bf16", f"pre {power}", pre=kind, eps=0.0)
    out = _run(x, "bf16", "h", post=kind, eps=0.0)
    _check(out, xv, "bf16", f"post {power}", post=kind, eps=0.0)


def test_large_rows_with_opposite_signs():
    """Elements near the type's largest, sums and deviations beyond it."""
    K = 256
    for signs in (np.ones(K), np.where(np.arange(K) % 2, 1.0, -1.0), np.where(np.arange(K) < 3, -1.0, 1.0)):
        x, xv = device((signs * 3.0e38 * (1 - np.arange(K) / 1000.0))[None], "bf16")
        for kind in ("rms", "layer"):
            _check(_run(x, "bf16", "y", pre=kind, eps=1e-6), xv, "bf16", kind, pre=kind)


def test_constant_and_zero_rows():
    for value in (0.0, 1.0, -3.0, 2.0**70, 2.0**-70):
        x, xv = device(np.full((2, 1000), value), "bf16")
        y = values(_run(x, "bf16", "y", pre="layer")["y"])
        assert np.abs(y).max() <= 64 * U * abs(value) / 1e-3 + 1e-30      # the mean's rounding over sqrt(eps)
        y = values(_run(x, "bf16", "y", pre="rms")["y"])
        _check(_run(x, "bf16", "y", pre="rms"), xv, "bf16", str(value))
    out = _run(torch.zeros((3, 256), dtype=torch.float16, device="cuda"), "fp16", "hyq", pre="rms")
    assert not out["y"].any() and not out["q"].any() and not out["s"].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("K", [256, 6144])
def test_odd_values_stay_in_their_row(bad, K):
    x, xv, dev, _ = _case(4, K, 2, "bf16", 21)
    clean = _run(x, "bf16", "hy", post="rms", pre="rms", **dev)
    for name in ("x", "residual"):
        t = {**dev, "x": x}
        t[name] = t[name].clone()
        t[name][2, 5] = bad
        out = _run(t.pop("x"), "bf16", "hy", post="rms", pre="rms", **t)
        rows = [0, 1, 3]
        assert torch.equal(out["h"][rows], clean["h"][rows]) and torch.equal(out["y"][rows], clean["y"][rows])
        assert not np.isfinite(values(out["h"])[2]).all() and not np.isfinite(values(out["y"])[2]).all()


def test_codes_feed_the_linear():
    """The codes and scales are the FP8 linear's operand."""
    M, K, N = 9, 512, 256
    x, xv, dev, host = _case(M, K, 3, "bf16", 22)
    out = _run(x, "bf16", "q", pre="layer", **dev)
    rng = np.random.default_rng(23)
    wq = torch.from_numpy(rng.integers(0, 0x70, (N, K)).astype(np.uint8)).cuda()
    wsc = torch.from_numpy(rng.uniform(0.5, 2, (N // 128, K // 128)).astype(np.float32)).cuda()
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    B.fp8_linear(out["q"], out["s"], wq, wsc, Y)
    want, mag = O.fp8_linear(out["q"].cpu().numpy(), values(out["s"]), wq.cpu().numpy(), values(wsc))
    assert_within(values(Y), want, mag * 2.0**-18 + half_ulp(np.abs(want) + mag * 2.0**-18, "bf16"), "linear")
