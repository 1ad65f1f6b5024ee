"""Pins of the block oracle (oracle/block.py) and CPU tests of the host side
of the operators around the layer: the rotary frequency table and the
refusals of the C ABI (every argument is checked before any device call)."""
import ctypes as C

import numpy as np
import pytest

import rank_gemm_svdq_amd as B
from rank_gemm_svdq_amd import binding as BB
from oracle import block as O


def test_e4m3_values_and_rounding():
    v = O.e4m3_values()
    assert v[0x7E] == 448.0 and v[0x01] == 2.0**-9 and v[0x08] == 2.0**-6 and v[0x38] == 1.0 and v[0xB8] == -1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and np.isfinite(v).sum() == 254
    fine = np.flatnonzero(np.isfinite(v))
    assert np.array_equal(O.e4m3_encode(v[fine]), fine)                 # every value is its own nearest
    # ties: halfway between neighbours goes to the even code
    mid = (v[:126] + v[1:127]) / 2
    assert np.all(O.e4m3_encode(mid) % 2 == 0)
    x = np.random.default_rng(1).uniform(-448, 448, 4000)
    near = np.abs(x[:, None] - v[fine][None, :]).min(1)
    assert np.array_equal(np.abs(x - O.e4m3_decode(O.e4m3_encode(x))), near)


def test_norm_pins():
    h, y, s = O.add_rmsnorm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0, np.array([[0.0, 0.0]]))
    r = np.sqrt(12.5)
    assert np.allclose(y, [[3 / r, -8 / r]]) and np.allclose(s, 8 / r / 448)
    _, y, s = O.add_rmsnorm(np.ones((1, 130)) * 5, np.ones(130), 0.0)
    assert np.allclose(y, 1.0) and s.shape == (1, 2)
    _, y, s = O.add_rmsnorm(np.zeros((1, 8)), np.ones(8), 1e-6)
    assert not y.any() and not s.any()


def test_fp8_linear_pins():
    rng = np.random.default_rng(2)
    xq, wq = rng.integers(0, 120, (3, 256), np.uint8), rng.integers(0, 120, (144, 256), np.uint8)
    xs, ws = rng.uniform(0.5, 2, (3, 2)), rng.uniform(0.5, 2, (2, 2))
    y, mag = O.fp8_linear(xq, xs, wq, ws, np.arange(144.0))
    v = O.e4m3_values()
    for m, n in [(0, 0), (2, 127), (1, 128), (2, 143)]:
        want = sum(xs[m, k // 128] * ws[n // 128, k // 128] * v[xq[m, k]] * v[wq[n, k]] for k in range(256))
        assert np.isclose(y[m, n], want + n) and np.isclose(mag[m, n], abs(want))


def test_rope_is_a_complex_product():
    rng = np.random.default_rng(3)
    x, pos = rng.standard_normal((5, 2, 24)), rng.integers(0, 99, (5, 2))
    for shared in (False, True):
        t = O.rope_angles(pos, [4, 12], 100.0, shared)
        e = [0, 1 / 2, 0, 1 / 6, 2 / 6, 3 / 6, 4 / 6, 5 / 6] if not shared else [j / 8 for j in range(8)]
        assert np.allclose(t, pos[:, [0, 0, 1, 1, 1, 1, 1, 1]] * 100.0 ** -np.array(e))
        y, _ = O.rope(x, t, True)
        z = (x[..., 0:16:2] + 1j * x[..., 1:16:2]) * np.exp(1j * t)[:, None, :]
        assert np.allclose(y[..., 0:16:2], z.real) and np.allclose(y[..., 1:16:2], z.imag)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        y, _ = O.rope(x, t, False)
        z = (x[..., 0:8] + 1j * x[..., 8:16]) * np.exp(1j * t)[:, None, :]
        assert np.allclose(y[..., 0:8], z.real) and np.allclose(y[..., 8:16], z.imag)


def test_attention_pins():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((1, 3, 2, 8)), rng.standard_normal((1, 5, 1, 8)), rng.standard_normal((1, 5, 1, 8))
    # a huge scale picks the best visible key: causal, queries are positions 1, 2, 3 of 4 keys in use
    o, *_ = O.attention(q, k, v, 1e6, causal=True, kv_len=[4])
    for i in range(3):
        for h in range(2):
            j = np.argmax(k[0, :2 + i, 0] @ q[0, i, h])
            assert np.allclose(o[0, i, h], v[0, j, 0])
    # scale 0: the mean over visible keys; prefix and documents
    o, *_ = O.attention(q, k, v, 0.0, causal=True, prefix=[5])
    assert np.allclose(o[0, 0, 0], v[0, :, 0].mean(0))
    o, _, _, seen = O.attention(q, k, v, 0.0, q_doc=[[1, 2, 7]], k_doc=[[1, 1, 2, 2, 2]])
    assert np.allclose(o[0, 0, 0], v[0, :2, 0].mean(0)) and np.allclose(o[0, 1, 1], v[0, 2:, 0].mean(0))
    assert not o[0, 2].any() and seen[0, 2].tolist() == [0, 0]
    # the bias alone: weights exp(-slope |distance|)
    o, *_ = O.attention(q, k, v, 0.0, slopes=[0.5, 1.0])
    w = np.exp(-0.5 * np.abs(2 - np.arange(5)))
    assert np.allclose(o[0, 0, 0], w @ v[0, :, 0] / w.sum())
    # the cap: scores cannot differ by more than twice the cap
    o, *_ = O.attention(1e9 * q, k, v, 1.0, softcap=1e-9)
    assert np.allclose(o[0, 1, 1], v[0, :, 0].mean(0))


@pytest.mark.parametrize("dims,theta,shared", [([16, 56, 56], 10000.0, False), ([16, 24, 24], 1e6, True),
                                               ([128], 500.0, False), ([0, 16, 0, 32], 10000.0, False)])
def test_rope_frequencies_against_64_bits(dims, theta, shared):
    turns, axis = B.rope_frequencies(dims, theta, shared)
    want = O.rope_angles(np.ones((1, len(dims))), dims, theta, shared)[0] / (2 * np.pi)
    got = turns[:, 0].astype(np.float64) + turns[:, 1]
    assert np.all(np.abs(got - want) <= 2.0**-47 * want)
    assert axis.tolist() == [a for a, d in enumerate(dims) for _ in range(d // 2)]


@pytest.mark.parametrize("dims,theta,status", [([], 1e4, 2), ([2] * 9, 1e4, 2), ([15, 17], 1e4, 2), ([8], 1e4, 2),
                                               ([528], 1e4, 2), ([-16, 32], 1e4, 2), ([16], 0.0, 1),
                                               ([16], float("nan"), 1), ([16], float("inf"), 1), ([24], 1e4, 2)])
def test_rope_frequencies_refusals(dims, theta, status):
    with pytest.raises(B.SvdqError) as e:
        B.rope_frequencies(dims, theta)
    assert e.value.status == status


# Refusals of the device entry points.  The pointers are never followed: each
# call has one wrong argument, found before any device call.
P = 1 << 20     # an aligned address
ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.mark.parametrize("change,status", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(M=0), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(K=4), SHAPE), (dict(K=132), SHAPE),
    (dict(K=65544), SHAPE), (dict(xst=120), SHAPE), (dict(rst=0), SHAPE), (dict(hst=8), SHAPE),
    (dict(xst=129), ALIGN), (dict(rst=132), ALIGN), (dict(hst=130), ALIGN), (dict(x=P + 2), ALIGN),
    (dict(r=P + 8), ALIGN), (dict(w=P + 4), ALIGN), (dict(h=P + 2), ALIGN), (dict(q=P + 8), ALIGN),
    (dict(s=P + 2), ALIGN), (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED)])
def test_norm_refusals(change, status):
    a = dict(x=P, xst=128, r=P, rst=128, w=P, eps=1e-6, M=4, K=128, dtype=0, h=P, hst=128, q=P, s=P)
    a.update(change)
    assert B.lib().svdq_add_rmsnorm_quantize(a["x"], a["xst"], a["r"], a["rst"], a["w"], a["eps"], a["M"], a["K"],
                                             a["dtype"], a["h"], a["hst"], a["q"], a["s"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(xq=None), ARG), (dict(xs=None), ARG), (dict(wq=None), ARG), (dict(ws=None), ARG), (dict(Y=None), ARG),
    (dict(M=0), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(K=64), SHAPE), (dict(K=192), SHAPE),
    (dict(N=8), SHAPE), (dict(N=24), SHAPE), (dict(N=262160), SHAPE), (dict(M=1 << 20, K=8192), SHAPE),
    (dict(K=65536, N=262144), SHAPE), (dict(xq=P + 8), ALIGN), (dict(wq=P + 1), ALIGN), (dict(xs=P + 1), ALIGN),
    (dict(ws=P + 2), ALIGN), (dict(bias=P + 2), ALIGN), (dict(Y=P + 8), ALIGN), (dict(dtype=7), UNSUPPORTED)])
def test_fp8_linear_refusals(change, status):
    a = dict(xq=P, xs=P, wq=P, ws=P, bias=P, M=4, K=128, N=16, dtype=1, Y=P)
    a.update(change)
    assert B.lib().svdq_fp8_linear(a["xq"], a["xs"], a["wq"], a["ws"], a["bias"], a["M"], a["K"], a["N"], a["dtype"],
                                   a["Y"], None) == status


def test_fp8_linear_workspace_and_its_refusals():
    need = B.fp8_linear_workspace_bytes
    assert need(333, 12288, 3072) == 7 * 3 * 24 * 128 * 128 * 4
    assert all(need(M, K, N) == 0 for M, K, N in [(0, 12288, 3072), (333, 12300, 3072), (333, 12288, 3080), (1, 128, 16),
                                                  (1, 12288, 3072), (333, 4096, 3072), (8192, 12288, 3072)])
    for M in (1, 100, 128, 129, 333, 1000, 2049, 5000, 1 << 18):
        for K in (128, 6144, 8192, 12288, 16384):
            for N in (16, 400, 3072, 4112, 65536):
                assert need(M, K, N) <= 32 << 20
    a = dict(xq=P, xs=P, wq=P, ws=P, bias=P, M=333, K=12288, N=3072, dtype=1, Y=P, w=P, n=need(333, 12288, 3072))
    for change, status in [(dict(w=None), ARG), (dict(n=a["n"] - 1), WORKSPACE), (dict(w=P + 4), ALIGN),
                           (dict(xs=None), ARG), (dict(bias=P + 2), ALIGN), (dict(dtype=2), UNSUPPORTED),
                           (dict(M=0), SHAPE), (dict(M=1, w=None, n=0, Y=None), ARG)]:
        assert B.lib().svdq_fp8_linear_shared(*{**a, **change}.values(), None) == status, change


def _rope_args(**change):
    a = BB.RopeArgs(4, 3, 16, 64, 1, 0, P, P, P)
    a.x[0] = a.y[0] = a.x[1] = a.y[1] = P
    a.heads[0], a.heads[1] = 2, 1
    for t in (a.x_token, a.y_token):
        t[0] = t[1] = 192
    for t in (a.x_head, a.y_head):
        t[0] = t[1] = 64
    for k, v in change.items():
        if k[-1] in "01" and k[:-1] in ("x", "y", "heads", "x_token", "x_head", "y_token", "y_head"):
            getattr(a, k[:-1])[int(k[-1])] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(positions=None), ARG), (dict(turns=None), ARG), (dict(axis=None), ARG), (dict(x0=None), ARG),
    (dict(y0=None), ARG), (dict(x1=None), ARG), (dict(y1=None), ARG), (dict(M=0), SHAPE), (dict(axes=0), SHAPE),
    (dict(axes=9), SHAPE), (dict(pairs=0), SHAPE), (dict(pairs=12), SHAPE), (dict(pairs=40), SHAPE),
    (dict(head_dim=520), SHAPE), (dict(head_dim=60), SHAPE), (dict(heads0=0), SHAPE), (dict(heads1=-1), SHAPE),
    (dict(heads0=65536), SHAPE), (dict(x0=P + 2), ALIGN), (dict(y1=P + 8), ALIGN), (dict(positions=P + 2), ALIGN),
    (dict(x_token0=4), ALIGN), (dict(y_head1=65), ALIGN), (dict(y_token0=256), ARG), (dict(dtype=3), UNSUPPORTED)])
def test_rope_refusals(change, status):
    assert B.lib().svdq_rope(C.byref(_rope_args(**change)), None) == status


def test_null_argument_structs():
    assert B.lib().svdq_rope(None, None) == ARG
    assert B.lib().svdq_attention(None, None, 0, None) == ARG


def _attn_args(**change):
    a = BB.AttentionArgs(2, 3, 5, 4, 2, 64, 0, 1, 0.125, 0.0, P, P, P, P, *[64 * 8, 64 * 4, 64] * 4)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(q=None), ARG), (dict(o=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(B=0), SHAPE),
    (dict(Sq=0), SHAPE), (dict(Skv=-1), SHAPE), (dict(Skv=(1 << 24) + 1), SHAPE), (dict(Hq=0), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(Hkv=3), SHAPE), (dict(Hkv=8), SHAPE), (dict(D=4), SHAPE), (dict(D=68), SHAPE),
    (dict(D=136), SHAPE), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(softcap=-1.0), ARG), (dict(softcap=float("inf")), ARG), (dict(softcap=float("nan")), ARG),
    (dict(q_doc=P), ARG), (dict(k_doc=P), ARG), (dict(q=P + 2), ALIGN), (dict(k=P + 8), ALIGN), (dict(o=P + 4), ALIGN),
    (dict(q_head=68), ALIGN), (dict(v_token=4), ALIGN), (dict(o_batch=1), ALIGN), (dict(kv_len=P + 2), ALIGN),
    (dict(slopes=P + 1), ALIGN), (dict(prefix=P + 3), ALIGN), (dict(dtype=2), UNSUPPORTED)])
def test_attention_refusals(change, status):
    assert B.lib().svdq_attention(C.byref(_attn_args(**change)), P, 1 << 40, None) == status
