"""Attention against the 64-bit oracle.

Bound.  With u = 2^-24: a score is off by (2 D + 16) u times its magnitudes
(products summed in the matrix unit, the cap's tanh through an exponential,
the bias), so a weight by e^2d - 1 < 3 d relative with d that error plus 2^-21
for the exponential; rounding the weights to the call's type adds 2^-8 (bf16)
or 2^-11 (fp16); adding n weighted values in fp32 adds 2 n u at most.  All of
these are relative to mean |v| + |o|.  Weights below fp16's range (the running
maximum may lag by 2^8) lose at most 2^-25 each: n 2^-25 max |v|.  The store
adds half an ulp."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import block as O
from tests.block_util import DTYPES, assert_within, device, half_ulp, values

pytestmark = pytest.mark.gpu


def _bound(o, mean, weight, seen, D, kind, vmax):
    u = 2.0**-24
    d = (2 * D + 16) * u * weight[..., None] + 2.0**-21
    n = seen[..., None]
    rel = 3 * d + (2.0**-8 if kind == "bf16" else 2.0**-11) + 2 * n * u
    e = rel * (mean + np.abs(o)) + (n * 2.0**-25 * vmax if kind == "fp16" else 0.0)
    return np.where(n > 0, e + half_ulp(np.abs(o) + e, kind), 0.0)


def _gpu(q, k, v, ws=None, stream=None, **kw):
    o = torch.full_like(q, float("nan"), memory_format=torch.contiguous_format)
    ws = B.attention_workspace(q, k) if ws is None else ws
    ints = {n: torch.from_numpy(np.asarray(kw[n], np.int32)).cuda() for n in ("kv_len", "prefix", "q_doc", "k_doc")
            if kw.get(n) is not None}
    sl = None if kw.get("slopes") is None else torch.from_numpy(np.asarray(kw["slopes"], np.float32)).cuda()
    rest = {n: kw[n] for n in ("scale", "causal", "softcap") if n in kw}
    B.attention(q, k, v, o, ws, slopes=sl, stream=stream, **rest, **ints)
    torch.cuda.synchronize()
    return o


def _make(B_, Sq, Skv, Hq, Hkv, D, kind, seed, gain=1.5):
    rng = np.random.default_rng(seed)
    return (device(gain * rng.standard_normal((B_, Sq, Hq, D)), kind),
            device(gain * rng.standard_normal((B_, Skv, Hkv, D)), kind),
            device(rng.standard_normal((B_, Skv, Hkv, D)), kind))


def _check(o, qv, kv, vv, kind, what, **kw):
    D = qv.shape[-1]
    kw = dict(kw)
    kw.setdefault("scale", D ** -0.5)
    if kw.get("slopes") is not None:
        kw["slopes"] = np.asarray(kw["slopes"], np.float32)
    want, mean, weight, seen = O.attention(qv, kv, vv, **kw)
    fine = np.abs(vv[np.isfinite(vv)]).max(initial=0.0)
    assert_within(values(o), want, _bound(want, mean, weight, seen, D, kind, fine), what)


SHAPES = [  # B, Sq, Skv, Hq, Hkv, D
    (1, 1, 1, 1, 1, 8), (1, 1, 2, 2, 1, 64), (2, 1, 33, 4, 2, 128), (3, 1, 64, 8, 1, 64), (1, 1, 65, 24, 8, 128),
    (2, 1, 1000, 6, 2, 128), (1, 1, 4099, 5, 1, 64), (2, 2, 77, 3, 3, 128), (1, 5, 300, 16, 2, 72), (1, 8, 8, 2, 2, 16),
    (1, 17, 130, 12, 4, 64), (2, 31, 31, 2, 1, 128), (1, 33, 96, 3, 1, 40), (1, 64, 64, 1, 1, 64), (1, 65, 129, 2, 2, 128),
    (1, 127, 200, 4, 1, 104), (1, 129, 257, 2, 1, 64), (2, 200, 511, 2, 2, 128), (1, 300, 300, 7, 7, 120), (1, 513, 700, 1, 1, 128)]


# blocks of 128 rows: enough of them, or many rows times keys (the last: in parts)
MANY = [(13, 129, 131, 8, 8, 64), (7, 129, 257, 8, 8, 128), (6, 129, 200, 16, 8, 104), (2, 513, 520, 16, 16, 40),
        (1, 700, 2100, 4, 4, 64)]


@pytest.mark.parametrize("shape", SHAPES + MANY)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["all", "causal", "causal_cap", "slopes", "len", "docs", "prefix", "everything"])
def test_against_oracle(shape, kind, mode):
    B_, Sq, Skv, Hq, Hkv, D = shape
    rng = np.random.default_rng(sum(shape))
    (q, qv), (k, kv), (v, vv) = _make(*shape, kind, sum(shape) + 1)
    kw = {}
    if mode != "all" and mode not in ("len", "docs", "slopes"):
        kw["causal"] = True
    if mode in ("causal_cap", "everything"):
        kw["softcap"] = 5.0
    if mode in ("slopes", "everything"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq)
    if mode in ("len", "everything"):
        kw["kv_len"] = rng.integers(0, Skv + 1, B_)          # shorter than Sq too: rows that see nothing
    if mode in ("prefix", "everything"):
        kw["prefix"] = rng.integers(-1, Skv + 2, B_)
    if mode in ("docs", "everything"):
        kw["k_doc"] = np.sort(rng.integers(-2, 3, (B_, Skv)), axis=1)
        kw["q_doc"] = rng.integers(-2, 4, (B_, Sq)) if mode == "docs" else kw["k_doc"][:, -Sq:]
    o = _gpu(q, k, v, **kw)
    _check(o, qv, kv, vv, kind, f"{mode} {shape}", **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("Sq,Skv,Hq,Hkv", [(1, 600, 4, 2), (3, 200, 2, 1), (150, 400, 2, 1), (40, 40, 1, 1),
                                             (150, 400, 104, 52)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_hidden_keys_may_hold_anything(kind, Sq, Skv, Hq, Hkv, bad):
    """NaN, infinities and the type's lowest value where a query does not look: past kv_len, in other documents,
    after the query; the outputs are those of clean caches."""
    D, B_ = 64, 2
    (q, qv), (k, kv), (v, vv) = _make(B_, Sq, Skv, Hq, Hkv, D, kind, 21)
    n = [Skv - 7, max(Sq, Skv // 3)]
    k_doc = np.zeros((B_, Skv), np.int32)
    k_doc[:, 5:30] = 1                              # seen by nobody
    k_doc[0, Skv - 20:Skv - 17] = 2
    q_doc = np.zeros((B_, Sq), np.int32)
    dirty_k, dirty_v = k.clone(), v.clone()
    lowest = torch.finfo(DTYPES[kind]).min
    for t in (dirty_k, dirty_v):
        t[:, 5:30] = bad
        t[0, Skv - 20:Skv - 17] = lowest
        for b in range(B_):
            t[b, n[b]:] = bad
    kw = dict(kv_len=n, causal=True, k_doc=k_doc, q_doc=q_doc)
    o = _gpu(q, dirty_k, dirty_v, **kw)
    clean = _gpu(q, k, v, **kw)
    _check(clean, qv, kv, vv, kind, "clean", **kw)
    _check(o, qv, kv, vv, kind, "dirty", **kw)
    # a key after some queries and before others: only the latter become what it holds
    if Sq > 2:
        at = n[0] - 2                               # position of the last query but one
        dirty_v[0, at] = float("nan")
        o = values(_gpu(q, k, dirty_v, **kw))
        assert np.isnan(o[0, Sq - 2:]).all() and np.isfinite(o[0, :Sq - 2]).all() and np.isfinite(o[1]).all()


def test_no_keys_at_all():
    (q, _), _, _ = _make(2, 3, 4, 2, 1, 64, "bf16", 1)
    k = torch.empty((2, 0, 1, 64), dtype=torch.bfloat16, device="cuda")
    assert not _gpu(q, k, k).any()
    assert not _gpu(q, k, k, causal=True, kv_len=[0, 5]).any()
    k = torch.full((2, 9, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert not _gpu(q, k, k, kv_len=[0, -3]).any()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("Sq,Skv,H", [(1, 2000, 2), (200, 200, 2), (200, 200, 160)])
def test_extreme_scores(kind, Sq, Skv, H):
    """Scores far apart (one key takes all), equal scores, scores whose maximum climbs along the keys and one whose
    exponentials would overflow without the maximum."""
    D = 64
    (q, qv), (k, kv), (v, vv) = _make(1, Sq, Skv, H, H // 2, D, kind, 31)
    for gain in (40.0, 0.0, 1e-3):
        _check(_gpu(q, k, v, scale=gain), qv, kv, vv, kind, f"scale {gain}", scale=gain)
    up = np.linspace(0, 1, Skv)[None, :, None, None] * np.ones((1, Skv, H // 2, D))
    kd, kdv = device(up, kind)
    qd, qdv = device(np.ones((1, Sq, H, D)), kind)
    for scale in (4.0, -4.0):
        _check(_gpu(qd, kd, v, scale=scale), qdv, kdv, vv, kind, f"climbing {scale}", scale=scale)
    _check(_gpu(q, k, v, softcap=0.25, scale=40.0), qv, kv, vv, kind, "cap", softcap=0.25, scale=40.0)
    # scores of tens of thousands below zero everywhere: no row is empty
    sl = [200.0, 100.0] * (H // 2)
    _check(_gpu(q, k, v, slopes=sl, kv_len=[Skv]), qv, kv, vv, kind, "far", slopes=sl, kv_len=[Skv])
    qdoc, kdoc = np.zeros((1, Sq), np.int32), np.ones((1, Skv), np.int32)
    kdoc[0, 0] = 0                                  # the farthest key is the only one
    _check(_gpu(q, k, v, slopes=sl, q_doc=qdoc, k_doc=kdoc), qv, kv, vv, kind, "farthest only", slopes=sl,
           q_doc=qdoc, k_doc=kdoc)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("Sq", [1, 3, 140])
def test_strides(kind, Sq):
    """Q, K, V as columns of one projection; K and V with heads outermost; O inside a wider row."""
    B_, Skv, Hq, Hkv, D = 2, 150, 4, 2, 64
    rng = np.random.default_rng(41)
    qkv, x = device(rng.standard_normal((B_, Skv, Hq + 2 * Hkv, D)), kind)
    q, k, v = qkv[:, Skv - Sq:, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    want = dict(causal=True)
    o = torch.zeros((B_, Sq, Hq, 2 * D), dtype=q.dtype, device="cuda")
    B.attention(q, k, v, o[..., D:], B.attention_workspace(q, k), causal=True)
    _check(o[..., D:], values(q), values(k), values(v), kind, "columns", **want)
    assert not o[..., :D].any()
    kc = torch.full((B_, Hkv, 300, D + 8), float("nan"), dtype=q.dtype, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    kc[:, :, :Skv, :D] = k.transpose(1, 2)
    vc[:, :, :Skv, 8:] = v.transpose(1, 2)
    kt, vt = kc[..., :D].transpose(1, 2), vc[..., 8:].transpose(1, 2)
    o2 = _gpu(q, kt, vt, causal=True, kv_len=[Skv, Skv - 11])
    kv = values(kt)[:, :Skv], values(vt)[:, :Skv]
    _check(o2[:1], values(q)[:1], kv[0][:1], kv[1][:1], kind, "heads outermost", **want)
    _check(o2[1:], values(q)[1:], kv[0][1:, :Skv - 11], kv[1][1:, :Skv - 11], kind, "heads outermost, shorter", **want)


def test_strides_of_many_rows():
    B_, Sq, Skv, Hq, Hkv, D = 3, 140, 150, 64, 32, 64
    qkv, x = device(np.random.default_rng(42).standard_normal((B_, Skv, Hq + 2 * Hkv, D)), "bf16")
    q, k, v = qkv[:, Skv - Sq:, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    kt, vt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    for a, b in ((k, v), (kt, vt)):
        o = torch.zeros((B_, Sq, Hq, 2 * D), dtype=q.dtype, device="cuda")
        B.attention(q, a, b, o[..., D:], B.attention_workspace(q, a), causal=True)
        _check(o[..., D:], values(q), values(k), values(v), "bf16", "columns", causal=True)
        assert not o[..., :D].any()


def test_broadcast_keys():
    """One batch entry's K and V for all (stride 0)."""
    (q, qv), (k, kv), (v, vv) = _make(3, 4, 50, 2, 1, 64, "bf16", 51)
    ke, ve = k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1)
    _check(_gpu(q, ke, ve), qv, np.repeat(kv[:1], 3, 0), np.repeat(vv[:1], 3, 0), "bf16", "broadcast")


@pytest.mark.parametrize("Sq", [1, 100, 16500])
def test_offsets_past_32_bits(Sq):
    """Keys more than 2^32 bytes apart."""
    D, Skv = 64, 150
    step = (1 << 31) // 100 + 8 - ((1 << 31) // 100) % 8
    (q, qv), (k, kv), (v, vv) = _make(1, Sq, Skv, 1, 1, D, "bf16", 61)
    flat = torch.empty(step * Skv, dtype=torch.bfloat16, device="cuda")
    kb, vb = flat.as_strided((1, Skv, 1, D), (0, step, D, 1)), flat.as_strided((1, Skv, 1, D), (0, step, D, 1), D)
    kb.copy_(k)
    vb.copy_(v)
    assert (Skv - 1) * step * 2 > 1 << 32
    causal = Sq <= Skv
    _check(_gpu(q, kb, vb, causal=causal), qv, kv, vv, "bf16", "far apart", causal=causal)


def test_long_cache_on_sampled_heads():
    """A long cache, many splits: two entries of ragged length."""
    B_, Skv, Hq, Hkv, D = 2, 40001, 8, 2, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = mk(B_, 1, Hq, D) * 2, mk(B_, Skv, Hkv, D), mk(B_, Skv, Hkv, D)
    n = [40001, 12345]
    o = _gpu(q, k, v, kv_len=n, causal=True)
    for h in (0, 5):
        hk = h // 4
        _check(o[:, :, h:h + 1], values(q[:, :, h:h + 1]), values(k[:, :, hk:hk + 1]), values(v[:, :, hk:hk + 1]),
               "bf16", f"head {h}", kv_len=n, causal=True)


def test_documents_in_a_long_row_on_sampled_queries():
    """Enough blocks that none shares its keys, and more key tiles than a block looks through beforehand; documents in
    no order, one of them only at the far end."""
    Sq, Skv, H, D = 1024, 140000, 64, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.float16)
    q, k, v = mk(1, Sq, H, D), mk(1, Skv, H, D), mk(1, Skv, H, D)
    rng = np.random.default_rng(9)
    k_doc = np.full((1, Skv), 99, np.int32)
    k_doc[0, rng.integers(0, Skv, 3000)] = 1
    k_doc[0, 500:900] = 2
    k_doc[0, Skv - 700:] = 3
    q_doc = np.repeat(np.array([1, 2, 3, 4, 2, 3, 1, 3], np.int32), Sq // 8)[None]
    o = _gpu(q, k, v, q_doc=q_doc, k_doc=k_doc)
    for i, h in [(0, 0), (127, 63), (128, 5), (300, 17), (383, 63), (400, 2), (640, 30), (1023, 31)]:
        _check(o[:, i:i + 1, h:h + 1], values(q[:, i:i + 1, h:h + 1]), values(k[:, :, h:h + 1]), values(v[:, :, h:h + 1]),
               "fp16", f"query {i} head {h}", q_doc=q_doc[:, i:i + 1], k_doc=k_doc)
    assert not o[:, 384:512].any()                  # document 4 has no keys


@pytest.mark.parametrize("B_,Sq,Hq,Hkv,Skv", [(1, 1, 8, 8, 9000), (3, 5, 6, 1, 5000), (1, 90, 3, 1, 6000)])
def test_parts_that_see_nothing(B_, Sq, Hq, Hkv, Skv):
    """Keys split over blocks where the length, the mask and the documents leave whole parts empty."""
    D = 64
    (q, qv), (k, kv), (v, vv) = _make(B_, Sq, Skv, Hq, Hkv, D, "bf16", 111)
    n = [min(Skv, 700 + 10 * b) for b in range(B_)]
    _check(_gpu(q, k, v, kv_len=n, causal=True), qv, kv, vv, "bf16", "short", kv_len=n, causal=True)
    k_doc, q_doc = np.zeros((B_, Skv), np.int32), np.ones((B_, Sq), np.int32)
    k_doc[:, 4321:4330] = 1
    q_doc[:, Sq // 2:Sq // 2 + 1] = 7               # and one query without any key
    kw = dict(q_doc=q_doc, k_doc=k_doc)
    _check(_gpu(q, k, v, **kw), qv, kv, vv, "bf16", "nine keys", **kw)


def test_token_strides_out_of_range_are_refused():
    from tests.test_oracle_block import _attn_args
    import ctypes as C
    for change in (dict(k_token=(1 << 25) + 8), dict(v_token=-8), dict(k_token=-8), dict(v_token=(1 << 25) + 8)):
        assert B.lib().svdq_attention(C.byref(_attn_args(**change)), None, 0, None) == 2


@pytest.mark.parametrize("shape", [(1, 1, 5000, 8, 2, 128), (1, 260, 1300, 2, 1, 128), (2, 33, 500, 4, 2, 64)])
def test_same_bits_again_with_a_used_workspace(shape):
    (q, qv), (k, kv), (v, vv) = _make(*shape, "bf16", 71)
    ws = B.attention_workspace(q, k)
    first = _gpu(q, k, v, ws, causal=True)
    ws.fill_(0xFF)                                  # NaN everywhere
    again = _gpu(q, k, v, ws, causal=True)
    _gpu(q * 3, k, v, ws, kv_len=[7] * shape[0])
    assert torch.equal(first, again) and torch.equal(first, _gpu(q, k, v, ws, causal=True))


def test_replays_of_a_graph():
    (q, qv), (k, kv), (v, vv) = _make(2, 1, 3000, 8, 2, 128, "bf16", 81)
    ws = B.attention_workspace(q, k)
    n = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    call = lambda: B.attention(q, k, v, o, ws, causal=True, kv_len=n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([3000, 1234], [17, 2999], [0, 1], [2048, 64]):     # lengths change between replays
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        want = _gpu(q, k, v, causal=True, kv_len=lens)
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), lens
    del g


def test_two_streams_with_a_workspace_each():
    (q, _), (k, _), (v, _) = _make(2, 1, 4000, 8, 2, 128, "bf16", 91)
    want = _gpu(q, k, v)
    torch.cuda.synchronize()
    outs, keep = [], []
    for _ in range(2):
        s, ws, o = torch.cuda.Stream(), B.attention_workspace(q, k), torch.empty_like(q)
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            B.attention(q, k, v, o, ws, stream=s)
        outs.append(o)
        keep.append((s, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_refusals():
    (q, _), (k, _), (v, _) = _make(2, 1, 3000, 4, 2, 64, "bf16", 101)
    o, ws = torch.zeros_like(q), B.attention_workspace(q, k)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    good = dict(q=q, k=k, v=v, o=o, ws=ws)
    for change in [dict(q=q.float()), dict(q=q.cpu()), dict(k=k.half()), dict(v=v[:, :5]), dict(o=o[:, :, :2]), dict(o=o.half()),
                   dict(k=k[:1], v=v[:1]), dict(k=k[..., :32], v=v[..., :32]), dict(q=q[0]), dict(q=q[:, :, :3], o=o[:, :, :3]),
                   dict(kv_len=i32(3)), dict(kv_len=i32(2).long()), dict(prefix=i32(1)), dict(q_doc=i32(2, 1)),
                   dict(k_doc=i32(2, 3000)), dict(q_doc=i32(2, 2), k_doc=i32(2, 3000)), dict(slopes=torch.zeros(3, device="cuda")),
                   dict(slopes=torch.zeros(4, device="cuda", dtype=torch.float64)), dict(softcap=-1.0), dict(scale=float("nan")),
                   dict(ws=ws.float()), dict(q=q[..., ::2], k=k[..., :32], v=v[..., :32], o=o[..., :32])]:
        a = dict(good)
        a.update(change)
        with pytest.raises(B.SvdqError):
            B.attention(**a)
    if ws.numel():
        for small, status in ((ws[:-256], 5), (None, 1)):
            with pytest.raises(B.SvdqError) as e:
                B.attention(q, k, v, o, small)
            assert e.value.status == status
    assert not o.any()
