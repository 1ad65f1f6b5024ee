"""What the binding refuses of the paged cache's, paged attention's and the gated norm's tensors, before any launch; and
that a KVCache keeps the memory that it goes by."""
import copy
import pickle

import pytest
import torch

import rank_gemm_svdq_amd as B
from tests.serving_util import ints, random_cache, random_table

pytestmark = pytest.mark.gpu

ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5
PAGES, HEADS, PAGE, D, REQ, T = 6, 2, 16, 32, 2, 3


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def refused(status, fn, *args, **kw):
    with pytest.raises(B.SvdqError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)


def test_caches():
    k = torch.zeros((PAGES, HEADS, PAGE, D), dtype=torch.int8, device="cuda")
    v = torch.zeros((PAGES, HEADS, D, PAGE), dtype=torch.int8, device="cuda")
    s = torch.zeros((PAGES, HEADS, PAGE), device="cuda")
    B.KVCache(k, v, s, s.clone())
    refused(ARG, B.KVCache, k, v)                                    # codes without scales
    refused(ARG, B.KVCache, k, v, s)
    refused(ARG, B.KVCache, k, v, s, s.half())
    refused(ARG, B.KVCache, k, v.float(), s, s)
    refused(ARG, B.KVCache, k.float(), v.float(), s, s)
    refused(ARG, B.KVCache, k.bfloat16(), v.bfloat16(), s, s)        # values with scales
    refused(SHAPE, B.KVCache, k, k, s, s)
    refused(SHAPE, B.KVCache, k[0], v, s, s)
    refused(SHAPE, B.KVCache, k, v, s[:-1], s)
    refused(ARG, B.KVCache, k.transpose(1, 2).contiguous().transpose(1, 2), v, s, s)
    refused(ARG, B.KVCache, k, v.cpu(), s, s)
    wide = torch.zeros((PAGES, HEADS + 2, PAGE), device="cuda")
    refused(ARG, B.KVCache, k, v, wide[:, :HEADS], s)                # scales of two strides


def call_args():
    cache = random_cache(PAGES, HEADS, PAGE, D, "int8", "bf16", 1)
    table = ints(random_table(REQ, T, PAGES, 1))
    return cache, table, ints([5, 48])


@pytest.mark.parametrize("what, status", [
    ("k type", ARG), ("k and v type", ARG), ("k shape", SHAPE), ("v on the host", ARG), ("table type", ARG),
    ("table dims", SHAPE), ("position type", ARG), ("position count", SHAPE), ("entry strided", ARG), ("strides", ALIGN),
    ("no entry, more tokens than requests", SHAPE), ("cache", ARG)])
def test_writes(what, status):
    cache, table, _ = call_args()
    M = 3
    a = dict(table=table, position=ints([1, 2, 3]), k=bf16(M, HEADS, D), v=bf16(M, HEADS, D), entry=ints([0, 1, 0]))
    B.cache_write(cache, **a)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    if what == "k type": a["k"] = a["k"].half()
    if what == "k and v type": a.update(k=a["k"].float(), v=a["v"].float())
    if what == "k shape": a["k"] = bf16(M, HEADS + 1, D)
    if what == "v on the host": a["v"] = a["v"].cpu()
    if what == "table type": a["table"] = table.long()
    if what == "table dims": a["table"] = table[0]
    if what == "position type": a["position"] = a["position"].long()
    if what == "position count": a["position"] = ints([1, 2])
    if what == "entry strided": a["entry"] = ints([0, 0, 1, 1, 0, 0])[::2]
    if what == "strides": a["k"] = bf16(M, HEADS, D + 4)[:, :, :D]
    if what == "no entry, more tokens than requests": a["entry"] = None
    if what == "cache": cache = B.KVCache(bf16(PAGES, HEADS, PAGE, D).half(), bf16(PAGES, HEADS, D, PAGE).half())
    refused(status, B.cache_write, cache, **a)
    if what != "cache":
        assert all(torch.equal(x, y) for x, y in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


@pytest.mark.parametrize("what, status", [
    ("k shape", SHAPE), ("heads", SHAPE), ("requests", SHAPE), ("v type", ARG), ("kv_len type", ARG), ("start count", SHAPE),
    ("strides", ALIGN), ("values of another type", ARG)])
def test_reads(what, status):
    cache, table, n = call_args()
    a = dict(table=table, kv_len=n, k=bf16(REQ, 48, HEADS, D), v=bf16(REQ, 48, HEADS, D), start=None)
    B.cache_read(cache, **a)
    if what == "k shape": a["k"] = bf16(REQ, 47, HEADS, D)
    if what == "heads": a.update(k=bf16(REQ, 48, 1, D), v=bf16(REQ, 48, 1, D))
    if what == "requests": a["table"] = table[:1]
    if what == "v type": a["v"] = a["v"].half()
    if what == "kv_len type": a["kv_len"] = n.float()
    if what == "start count": a["start"] = ints([0])
    if what == "strides": a["v"] = bf16(REQ, 48, HEADS, D + 4)[..., :D]
    if what == "values of another type":
        cache = B.KVCache(bf16(PAGES, HEADS, PAGE, D).half(), bf16(PAGES, HEADS, D, PAGE).half())
    refused(status, B.cache_read, cache, **a)


@pytest.mark.parametrize("what, status", [
    ("heads", SHAPE), ("head size", SHAPE), ("o type", ARG), ("q type", ARG), ("kv_len count", SHAPE), ("slopes type", ARG),
    ("lse shape", SHAPE), ("negative window", ARG), ("negative cap", ARG), ("scale", ARG), ("workspace type", ARG),
    ("no workspace", ARG), ("small workspace", WORKSPACE), ("workspace off its alignment", ALIGN), ("cache", ARG)])
def test_paged_attention(what, status):
    cache = random_cache(600, HEADS, PAGE, D, "int8", "bf16", 1)
    table, n = ints(random_table(REQ, 300, 600, 1)), ints([7, 4800])
    a = dict(table=table, kv_len=n, q=bf16(REQ, 8, D), o=bf16(REQ, 8, D))
    a["ws"] = B.paged_attention_workspace(a["q"], cache, table)
    assert a["ws"].numel() > 256                                     # parts to join
    B.paged_attention(a.pop("q"), cache, **a)
    a["q"] = bf16(REQ, 8, D)
    if what == "heads": a.update(q=bf16(REQ, 7, D), o=bf16(REQ, 7, D))
    if what == "head size": a.update(q=bf16(REQ, 8, 16), o=bf16(REQ, 8, 16))
    if what == "o type": a["o"] = a["o"].half()
    if what == "q type": a["q"] = a["q"].float()
    if what == "kv_len count": a["kv_len"] = ints([7])
    if what == "slopes type": a["slopes"] = bf16(8)
    if what == "lse shape": a["lse"] = torch.zeros((8, REQ), device="cuda")
    if what == "negative window": a["window"] = -1
    if what == "negative cap": a["softcap"] = -1.0
    if what == "scale": a["scale"] = float("nan")
    if what == "workspace type": a["ws"] = a["ws"].float()
    if what == "no workspace": a["ws"] = None
    if what == "small workspace": a["ws"] = a["ws"][:-256]
    if what == "workspace off its alignment": a["ws"] = torch.cat((a["ws"], a["ws"]))[16:]
    if what == "cache": cache = "cache"
    if what == "cache":
        with pytest.raises(AttributeError):
            B.paged_attention(a.pop("q"), cache, **a)
    else:
        refused(status, B.paged_attention, a.pop("q"), cache, **a)


@pytest.mark.parametrize("what, status", [
    ("y type", ARG), ("residual shape", SHAPE), ("gate rows", SHAPE), ("gate and shift", SHAPE), ("entry type", ARG),
    ("weight shape", SHAPE), ("q alone", ARG), ("s shape", SHAPE), ("nothing to write", ARG), ("y is h", ARG),
    ("columns", SHAPE), ("eps", ARG)])
def test_gated_norm(what, status):
    M, K = 6, 128
    a = dict(x=bf16(M, K), y=bf16(M, K))
    B.gated_norm(**a)
    if what == "y type": a["y"] = a["y"].half()
    if what == "residual shape": a["residual"] = bf16(M + 1, K)
    if what == "gate rows": a["gate"] = bf16(4, K)                   # 6 rows in 4
    if what == "gate and shift": a.update(gate=bf16(2, K), shift=bf16(3, K))
    if what == "entry type": a.update(gate=bf16(2, K), entry=ints([0] * M).long())
    if what == "weight shape": a["weight"] = bf16(K - 8)
    if what == "q alone": a["q"] = torch.zeros((M, K), dtype=torch.float8_e4m3fn, device="cuda")
    if what == "s shape":
        a.update(q=torch.zeros((M, K), dtype=torch.float8_e4m3fn, device="cuda"), s=torch.zeros((M, 2), device="cuda"))
    if what == "nothing to write": a["y"] = None
    if what == "y is h": a["h"] = a["y"]
    if what == "columns": a.update(x=bf16(M, 132)[:, :130], y=bf16(M, 132)[:, :130])
    if what == "eps": a["eps"] = -1.0
    refused(status, B.gated_norm, **a)


def test_a_cache_keeps_its_memory():
    cache, table, n = call_args()
    with pytest.raises(AttributeError):
        cache.k = cache.k.clone()                                    # the calls would go on with the old one
    q = torch.randn((REQ, 4, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()

    def attend(c):
        o = torch.empty_like(q)
        B.paged_attention(q, c, table, n, o, B.paged_attention_workspace(q, c, table))
        return o
    want = attend(cache)
    assert want.float().abs().sum() > 0
    for other in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert other.k.data_ptr() != cache.k.data_ptr()
        other.k_scale.fill_(float("nan"))                            # its own
        assert torch.equal(attend(cache), want) and attend(other).isnan().all()
    shallow = copy.copy(cache)
    assert shallow.k is cache.k and torch.equal(attend(shallow), want)


def test_bits_of_bf16_are_bf16():
    """int16 tensors stand for the bits of bf16 ones, the cache's too."""
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((20, HEADS, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((1, 4, D), generator=g).to(torch.bfloat16).cuda()
    table, bits = ints([[3, 1]]), lambda t: t.view(torch.int16)
    got = []
    for view in (lambda t: t, bits):
        cache = B.KVCache(view(bf16(PAGES, HEADS, PAGE, D)), view(bf16(PAGES, HEADS, D, PAGE)))
        B.cache_write(cache, table, ints(range(20)), view(k), view(v), entry=ints([0] * 20))
        o, kr, vr = torch.empty_like(q), bf16(1, 20, HEADS, D), bf16(1, 20, HEADS, D)
        B.paged_attention(view(q), cache, table, ints([20]), view(o), B.paged_attention_workspace(q, cache, table))
        B.cache_read(cache, table, ints([20]), view(kr), view(vr))
        assert torch.equal(kr[0], k) and torch.equal(vr[0], v)
        got.append(o)
    assert got[0].float().abs().sum() > 0 and torch.equal(got[0], got[1])


def test_writes_of_two_streams_into_one_page():
    """Calls that overlap in time may write different places of the same page."""
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn((64, 40, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = ints([[2]])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for fmt in ("int8", "bf16"):
        whole, parts = (B.KVCache.empty(3, 40, 64, page=64, format=fmt) for _ in range(2))
        B.cache_write(whole, table, ints(range(64)), k, v, entry=ints([0] * 64))
        places = [ints(range(0, 29)), ints(range(29, 64))]
        entries = [ints([0] * 29), ints([0] * 35)]
        torch.cuda.synchronize()
        for s, at, e, lo, hi in zip(streams, places, entries, (0, 29), (29, 64)):
            B.cache_write(parts, table, at, k[lo:hi], v[lo:hi], entry=e, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(parts.k, whole.k) and torch.equal(parts.v, whole.v) and whole.v.float().abs().sum() > 0
