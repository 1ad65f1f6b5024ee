"""Pins of oracle/serving.py, and refusals of the paged cache's, paged attention's and the gated norm's entries (CPU:
every argument is checked before any device call; the pointers are never followed)."""
import ctypes as C

import numpy as np
import pytest

import rank_gemm_svdq_amd as B
from oracle import block as O
from oracle import serving as S
from rank_gemm_svdq_amd import binding as BB

P = 1 << 20     # an aligned address
ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


# ---------------------------------------------------------------- the oracle

def test_encode_pins():
    c, s = S.encode(np.array([[127.0, -127.0, 0.5, 1.5, -2.5, 63.49]]), "int8")
    assert s.tolist() == [1.0] and c.tolist() == [[127, -127, 0, 2, -2, 63]]         # ties to even
    c, s = S.encode(np.array([[448.0, 1.0, -18.0, 17.0]]), "fp8")
    assert s.tolist() == [1.0] and c.tolist() == [[448, 1, -18, 16]]
    c, s = S.encode(np.array([[449.0, 3.0], [0.0, 0.0], [224.0, 1.0], [224.5, 1.0]]), "fp8")
    assert s.tolist() == [2.0, 0.0, 0.5, 1.0] and c[0].tolist() == [224, 1.5] and c[2].tolist() == [448, 2]
    for fmt in ("int8", "fp8"):
        c, s = S.encode(np.array([[1.0, np.nan], [np.inf, 2.0]]), fmt)
        assert np.isnan(s).all() and not c.any()
        x = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32)
        c, s = S.encode(x, fmt)
        step = s[:, None] / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0**-4, s[:, None] * 2.0**-10)
        assert np.all(np.abs(c * s[:, None] - x) <= step * (1 + 1e-6)) and np.abs(c).max() <= (127 if fmt == "int8" else 448)
        assert np.abs(c).max(1).min() >= (127 if fmt == "int8" else 224)


def test_write_and_dense_are_inverse():
    rng = np.random.default_rng(2)
    c = {"k": np.zeros((4, 2, 16, 16)), "v": np.zeros((4, 2, 16, 16)), "ks": np.zeros((4, 2, 16)), "vs": np.zeros((4, 2, 16))}
    table = np.array([[3, 0], [1, -1]])
    entry, pos = np.array([0, 0, 1, 1, 0, 2]), np.array([0, 31, 5, 20, -1, 0])
    k, v = rng.integers(-127, 128, (2, 6, 2, 16)).astype(float)
    k[..., 0] = v[..., 0] = 127
    w = S.write(c, table, entry, pos, k, v, "int8")
    dk, dv, there = S.dense(w, table)
    for m, b, p in ((0, 0, 0), (1, 0, 31), (2, 1, 5)):
        assert np.array_equal(dk[b, p], k[m]) and np.array_equal(dv[b, p], v[m]) and there[b, p]
    assert (dk != 0).any(-1).sum() == 6 and not there[1, 16:].any() and not c["k"].any()


def test_paged_attention_pins():
    rng = np.random.default_rng(3)
    c = {"k": rng.standard_normal((3, 2, 16, 16)), "v": rng.standard_normal((3, 2, 16, 16))}
    q, table = rng.standard_normal((1, 4, 16)), np.array([[2, 0, 9]])
    k = np.concatenate([c["k"][2], c["k"][0]], 1)
    v = np.concatenate([c["v"][2].transpose(0, 2, 1), c["v"][0].transpose(0, 2, 1)], 1)
    for n, window in ((20, 0), (20, 6), (40, 0), (1, 0)):
        o, _, _, seen, lse = S.paged_attention(q, c, table, [n], 0.3, window=window)
        lo, hi = max(0, n - window) if window else 0, min(n, 32)
        for h in range(4):
            w = np.exp(0.3 * k[h // 2, lo:hi] @ q[0, h])
            assert np.allclose(o[0, h], w @ v[h // 2, lo:hi] / w.sum()) and np.isclose(lse[0, h], np.log(w.sum()))
        assert (seen == hi - lo).all()
    o, _, _, _, lse = S.paged_attention(q, c, table, [0], 0.3)
    assert not o.any() and np.isneginf(lse).all()


def test_gated_norm_pins():
    x, r = np.array([[3.0, -4.0]]), np.array([[1.0, 1.0]])
    h, y = S.gated_norm(x, r, 2.0, post="rms", gate=np.array([[2.0, 0.5]]), pre="none", entry=np.array([0]), eps=0.0)
    s = np.sqrt(12.5)
    assert np.allclose(h, [[2 + 6 / s, 2 - 2 / s]]) and np.array_equal(h, y)
    h, y = S.gated_norm(np.array([[1.0, 3.0]]), pre="layer", scale=np.array([[0.0, 1.0]]), shift=np.array([[5.0, 0.0]]),
                        entry=np.array([0]), eps=0.0)
    assert np.allclose(y, [[4.0, 2.0]])
    _, y = S.gated_norm(np.array([[3.0, 4.0]]), weight=np.array([1.0, 2.0]), eps=0.0)
    assert np.allclose(y, O.add_rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)[1])


# ----------------------------------------------------------------- refusals

def _cache(**change):
    a = BB.KVCacheArgs(8, 64, 2, 128, 1, P, P, P, P, 2 * 64 * 128, 2 * 64 * 128, 2 * 64)
    for k, v in change.items():
        setattr(a, k, v)
    return a


CACHES = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG), (dict(pages=0), SHAPE),
          (dict(pages=(1 << 28) + 1), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE),
          (dict(heads=0), SHAPE), (dict(heads=65537), SHAPE), (dict(D=0), SHAPE), (dict(D=24), SHAPE), (dict(D=144), SHAPE),
          (dict(k_page=2 * 64 * 128 - 16), SHAPE), (dict(v_page=0), SHAPE), (dict(scale_page=2 * 64 - 4), SHAPE),
          (dict(k_page=-1), SHAPE), (dict(v_page=(1 << 34) + 16), SHAPE), (dict(k_page=2 * 64 * 128 + 8), ALIGN),
          (dict(v_page=2 * 64 * 128 + 1), ALIGN), (dict(scale_page=2 * 64 + 2), ALIGN), (dict(k=P + 8), ALIGN), (dict(v=P + 4), ALIGN),
          (dict(k_scale=P + 4), ALIGN), (dict(v_scale=P + 8), ALIGN), (dict(format=3), UNSUPPORTED), (dict(format=-1), UNSUPPORTED)]


def _write(cache=None, **change):
    a = BB.CacheWriteArgs(4, 4, 3, 0, P, 3, P, P, P, P, 256, 128, 256, 128)
    for k, v in change.items():
        setattr(a, k, v)
    return B.lib().svdq_cache_write(C.byref(cache or _cache()), C.byref(a), None)


def _read(cache=None, **change):
    a = BB.CacheReadArgs(4, 100, 3, 0, P, 3, P, P, P, P, 25600, 256, 128, 25600, 256, 128)
    for k, v in change.items():
        setattr(a, k, v)
    return B.lib().svdq_cache_read(C.byref(cache or _cache()), C.byref(a), None)


def _paged(cache=None, ws=P, bytes=1 << 40, **change):
    a = BB.PagedAttentionArgs(4, 3, 8, 0, 0, 0.1, 0.0, P, P, 1024, 128, 1024, 128, P, 3, P, P, P)
    for k, v in change.items():
        setattr(a, k, v)
    return B.lib().svdq_paged_attention(C.byref(cache or _cache()), C.byref(a), ws, bytes, None)


@pytest.mark.parametrize("change,status", CACHES)
def test_cache_refusals(change, status):
    for call in (_write, _read, _paged):
        assert call(_cache(**change)) == status, call.__name__
    if status != ARG and not any(k in ("k", "v", "k_scale", "v_scale") for k in change):
        assert B.lib().svdq_paged_attention_workspace_bytes(C.byref(_cache(**change)), 1, 1000, 8) == 0


def test_values_need_no_scales():
    c = _cache(format=0, k_scale=None, v_scale=None, scale_page=0)
    assert _write(c, M=0) == SHAPE and _read(c, S=0) == SHAPE and _paged(c, Hq=3) == SHAPE      # past the cache's checks
    assert _write(_cache(format=0, k_scale=None, v_scale=None, scale_page=0, k_page=2 * 64 * 128 + 4)) == ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(position=None), ARG), (dict(table=None), ARG), (dict(M=0), SHAPE),
    (dict(M=(1 << 20) + 1), SHAPE), (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(T=(1 << 18) + 1, table_row=1 << 20), SHAPE),
    (dict(table_row=2), SHAPE), (dict(M=5, entry=None), SHAPE), (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(entry=P + 1), ALIGN), (dict(position=P + 2), ALIGN), (dict(k_token=4), ALIGN),
    (dict(v_head=129), ALIGN), (dict(dtype=2), UNSUPPORTED)])
def test_write_refusals(change, status):
    assert _write(**change) == status


def test_more_blocks_than_a_launch_takes():
    big = _cache(heads=65536, page=16, D=16, k_page=1 << 24, v_page=1 << 24, scale_page=1 << 20)
    assert _write(big, M=1 << 20) == SHAPE and _read(big, S=1 << 20) == SHAPE and _read(big, B=1 << 30, S=1, table_row=3) == SHAPE
    assert _paged(big, Hq=65536, B=256, ws=None) == SHAPE


@pytest.mark.parametrize("change,status", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(kv_len=None), ARG), (dict(table=None), ARG), (dict(B=0), SHAPE),
    (dict(S=0), SHAPE), (dict(S=(1 << 24) + 1), SHAPE), (dict(T=0), SHAPE), (dict(table_row=2), SHAPE), (dict(k=P + 8), ALIGN),
    (dict(v=P + 2), ALIGN), (dict(table=P + 2), ALIGN), (dict(kv_len=P + 1), ALIGN), (dict(start=P + 2), ALIGN),
    (dict(k_batch=4), ALIGN), (dict(v_token=12), ALIGN), (dict(dtype=-1), UNSUPPORTED)])
def test_read_refusals(change, status):
    assert _read(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), ARG), (dict(o=None), ARG), (dict(kv_len=None), ARG), (dict(table=None), ARG), (dict(window=-1), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(softcap=-1.0), ARG), (dict(softcap=float("nan")), ARG),
    (dict(softcap=float("inf")), ARG), (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(T=(1 << 18) + 1, table_row=1 << 20), SHAPE),
    (dict(table_row=2), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=3), SHAPE), (dict(Hq=65538), SHAPE), (dict(B=1 << 21), SHAPE),
    (dict(q=P + 8), ALIGN), (dict(o=P + 2), ALIGN), (dict(q_batch=4), ALIGN), (dict(o_head=12), ALIGN), (dict(table=P + 2), ALIGN),
    (dict(kv_len=P + 1), ALIGN), (dict(slopes=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ws=P + 16), ALIGN),
    (dict(dtype=5), UNSUPPORTED)])
def test_paged_refusals(change, status):
    assert _paged(**change) == status


def test_paged_workspace():
    L, need = B.lib(), lambda c, *a: B.lib().svdq_paged_attention_workspace_bytes(C.byref(c), *a)
    assert L.svdq_paged_attention_workspace_bytes(None, 1, 1, 1) == 0
    assert need(_cache(), 0, 10, 8) == 0 and need(_cache(), 1, 10, 3) == 0 and need(_cache(), 1, (1 << 18) + 1, 8) == 0
    assert need(_cache(), 4, 3, 8) == 0                       # a short cache is one block's
    long = need(_cache(), 1, 1 << 12, 8)
    assert long > 0 and long % 256 == 0
    args = dict(B=1, T=1 << 12)
    assert _paged(ws=None, **args) == ARG and _paged(bytes=long - 1, **args) == WORKSPACE and _paged(ws=P + 4, **args) == ALIGN
    for B_ in (1, 2, 7, 100, 5000):                           # bounded, and enough for any window
        for T in (1, 16, 17, 100, 1000, 1 << 18):
            for page in (16, 64):
                c = _cache(page=page, k_page=1 << 20, v_page=1 << 20, scale_page=1 << 16)
                assert need(c, B_, T, 32) <= 256 << 20


def test_null_structs():
    L = B.lib()
    assert L.svdq_cache_write(None, None, None) == ARG and L.svdq_cache_read(C.byref(_cache()), None, None) == ARG
    assert L.svdq_paged_attention(None, None, None, 0, None) == ARG and L.svdq_gated_norm(None, None) == ARG


def _gated(**change):
    a = BB.GatedNormArgs(4, 256, 2, 0, 1, 2, 1e-6, 1.0, *[P] * 8, 2 * P, 3 * P, P, P, *[256] * 7)
    for k, v in change.items():
        setattr(a, k, v)
    return B.lib().svdq_gated_norm(C.byref(a), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), ARG), (dict(h=None, y=None, q=None, s=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(residual_scale=float("nan")), ARG),
    (dict(residual_scale=float("-inf")), ARG), (dict(y=2 * P), ARG), (dict(h=P, h_row=264), ARG), (dict(y=P, y_row=264), ARG),
    (dict(h=P, x_row=264, residual=5 * P), ARG), (dict(M=0), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(K=0), SHAPE),
    (dict(K=12), SHAPE), (dict(K=16392), SHAPE), (dict(E=0), SHAPE), (dict(E=(1 << 20) + 1), SHAPE), (dict(entry=None, E=3), SHAPE),
    (dict(x_row=248), SHAPE), (dict(residual_row=0), SHAPE), (dict(gate_row=8), SHAPE), (dict(scale_row=-256), SHAPE),
    (dict(shift_row=255), SHAPE), (dict(h_row=128), SHAPE), (dict(y_row=128), SHAPE), (dict(x_row=260), ALIGN),
    (dict(gate_row=257), ALIGN), (dict(y_row=258), ALIGN), (dict(x=P + 8), ALIGN), (dict(residual=P + 2), ALIGN),
    (dict(post_weight=P + 8), ALIGN), (dict(weight=P + 4), ALIGN), (dict(gate=P + 2), ALIGN), (dict(scale=P + 2), ALIGN),
    (dict(shift=P + 2), ALIGN), (dict(h=P + 2), ALIGN), (dict(y=2 * P + 2, h=None), ALIGN), (dict(q=P + 8), ALIGN),
    (dict(s=P + 2), ALIGN), (dict(entry=P + 2), ALIGN), (dict(dtype=2), UNSUPPORTED), (dict(post=3), UNSUPPORTED),
    (dict(pre=-1), UNSUPPORTED)])
def test_gated_refusals(change, status):
    assert _gated(**change) == status


def test_names_of_norms_and_formats():
    with pytest.raises(ValueError):
        B.gated_norm(None, pre="batch")
    with pytest.raises(ValueError):
        B.gated_norm(None, post="batch")
    with pytest.raises(ValueError):
        B.KVCache.empty(1, 1, 64, format="int4", device="cpu")


def test_tensors_are_checked():
    """What the binding says of wrong tensors, without a GPU: a cache's have to be in GPU memory."""
    torch = pytest.importorskip("torch")
    with pytest.raises(B.SvdqError) as e:
        B.KVCache.empty(2, 2, 64, device="cpu")
    assert e.value.status == ARG and "GPU" in str(e.value)
    with pytest.raises(B.SvdqError) as e:
        B.KVCache(1, 2)
    assert e.value.status == ARG
    with pytest.raises(B.SvdqError):
        B.gated_norm(torch.zeros((2, 8)), y=torch.zeros((2, 8)))
