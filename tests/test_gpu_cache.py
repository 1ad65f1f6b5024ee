"""Writing the paged cache and reading it back.

Codes and scales are defined to the bit (include/svdq.h), so a write is compared
for equality with the 64-bit oracle, and everything that a write does not name with
what was there.  A read is one fp32 product rounded to 16 bits: equal to the same in
torch."""
import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import serving as S
from tests.block_util import DTYPES, device, values
from tests.serving_util import ints, numpy_of, random_cache, random_table

pytestmark = pytest.mark.gpu


def _same(cache, want, what):
    got = numpy_of(cache)
    assert got.keys() == want.keys()
    for n in got:
        bad = ~((got[n] == want[n]) | (np.isnan(got[n]) & np.isnan(want[n])))
        assert not bad.any(), f"{what} {n}: {int(bad.sum())} of {bad.size} differ, first at {np.argwhere(bad)[0]}"


def _tokens(M, heads, D, kind, seed, strided=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, 3 * heads, D)) * np.where(rng.random(D) < 0.05, 8.0, 1.0)
    t, _ = device(x, kind)
    k, v = t[:, heads:2 * heads], t[:, 2 * heads:]
    return (k, v) if strided else (k.contiguous(), v.contiguous())


WRITES = [  # tokens, requests, heads, D, page, pages of a request
    (1, 1, 1, 16, 16, 1), (3, 3, 2, 128, 64, 2), (16, 16, 8, 128, 64, 3), (17, 2, 1, 64, 16, 4), (61, 1, 3, 80, 32, 4),
    (64, 1, 2, 128, 64, 2), (65, 4, 5, 96, 128, 1), (200, 3, 4, 112, 16, 9), (333, 2, 2, 48, 256, 2), (700, 1, 30, 64, 64, 13),
    (1100, 5, 24, 128, 64, 6),
    # enough tokens and heads for the kernel that turns values through LDS: odd sizes and scattered places too
    (130, 2, 48, 80, 32, 4), (200, 7, 40, 112, 16, 9), (301, 3, 32, 64, 16, 9), (65, 1, 64, 128, 64, 3), (640, 4, 13, 96, 128, 2),
    (129, 9, 43, 48, 256, 1)]


@pytest.mark.parametrize("shape", WRITES)
@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_write_against_oracle(shape, fmt, kind):
    M, B_, heads, D, page, T = shape
    rng = np.random.default_rng(sum(shape))
    cache = random_cache(B_ * T + 2, heads, page, D, fmt, kind, 1)
    table = random_table(B_, T, B_ * T + 2, 2)
    k, v = _tokens(M, heads, D, kind, 3)
    if M == B_:
        entry, pos = None, rng.integers(0, T * page, M)
    else:           # runs of positions from anywhere, some of them aligned
        at = rng.choice(B_ * T * page, M, replace=False) if M % 2 else np.arange(M) + rng.integers(0, B_ * T * page - M + 1)
        entry, pos = at // (T * page), at % (T * page)
        if M % 2:
            entry[::7], pos[::7] = -1, 0
            pos[1::9] = -5
    want = S.write(numpy_of(cache), table, entry, pos, values(k), values(v), fmt)
    B.cache_write(cache, ints(table), ints(pos), k, v, entry=None if entry is None else ints(entry))
    torch.cuda.synchronize()
    _same(cache, want, f"{shape} {fmt} {kind}")


@pytest.mark.parametrize("first", range(0, 9))
@pytest.mark.parametrize("fmt", ["int8", "values"])
@pytest.mark.parametrize("heads", [2, 64])
def test_runs_that_start_inside_a_group_of_places(first, fmt, heads):
    """Prompts from any place on, over the ends of pages."""
    cache = random_cache(6, heads, 32, 64, fmt, "bf16", 4)
    table = random_table(1, 6, 6, 5)
    k, v = _tokens(150, heads, 64, "bf16", 6)
    pos, entry = np.arange(150) + first, np.zeros(150)
    want = S.write(numpy_of(cache), table, entry, pos, values(k), values(v), fmt)
    B.cache_write(cache, ints(table), ints(pos), k, v, entry=ints(entry))
    _same(cache, want, f"first {first}")


def test_several_requests_with_runs_of_their_own_phase():
    """Ragged prompts one after the other, padded rows between and behind them."""
    cache = random_cache(40, 48, 16, 64, "int8", "bf16", 4)
    table = random_table(5, 8, 40, 5)
    entry, pos = [], []
    for e, (start, n) in enumerate(((3, 50), (0, 41), (14, 77), (5, 1), (9, 100))):
        entry += [e] * n + [0] * 5
        pos += list(range(start, start + n)) + [-1] * 5
    k, v = _tokens(len(pos), 48, 64, "bf16", 6)
    want = S.write(numpy_of(cache), table, np.array(entry), np.array(pos), values(k), values(v), "int8")
    B.cache_write(cache, ints(table), ints(pos), k, v, entry=ints(entry))
    _same(cache, want, "ragged")
    # the same tokens in an order without runs
    o = np.random.default_rng(7).permutation(len(pos))
    other = random_cache(40, 48, 16, 64, "int8", "bf16", 4)
    B.cache_write(other, ints(table), ints(np.array(pos)[o]), k[torch.from_numpy(o).cuda()], v[torch.from_numpy(o).cuda()],
                  entry=ints(np.array(entry)[o]))
    _same(other, want, "shuffled")


@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
@pytest.mark.parametrize("heads", [2, 130])
def test_places_that_do_not_exist_are_passed_over(fmt, heads):
    cache = random_cache(5, heads, 16, 32, fmt, "fp16", 7)
    table = np.array([[0, -1, 7], [2, 5, 4], [3, 2**31 - 1, -2**31]], np.int32)
    pos = np.array([0, 16, 33, 47, 48, 2**31 - 1, -1, -2**31, 3, 17, 40, 15, 31, 32, 0, 0])
    entry = np.array([0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 1, 2, 2, 2, 3, -1])
    k, v = _tokens(16, heads, 32, "fp16", 8)
    before = numpy_of(cache)
    want = S.write(before, table, entry, pos, values(k), values(v), fmt)
    assert len(S.places(table, entry, pos, 5, 16)) == 4
    B.cache_write(cache, ints(table), ints(pos), k, v, entry=ints(entry))
    _same(cache, want, fmt)
    # all of them
    B.cache_write(cache, ints(table), ints(np.full(16, -1)), k, v, entry=ints(entry))
    _same(cache, want, fmt)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [1, 130])
def test_vectors_of_any_magnitude(fmt, kind, heads):
    """Zeros, subnormals, the largest values, halfway quotients, infinities and NaN."""
    D, big = 64, torch.finfo(DTYPES[kind]).max
    rng = np.random.default_rng(9)
    rows = [np.zeros(D), np.full(D, -0.0), np.r_[127.0, np.arange(D - 1) - 31.5], np.r_[-127.0, np.arange(D - 1) / 2],
            np.r_[448.0, np.arange(D - 1) / 16], np.r_[450.0, rng.standard_normal(D - 1) * 30], np.full(D, big), np.full(D, -big),
            np.r_[big, np.full(D - 1, 1.0)], rng.standard_normal(D) * 2.0**-20, np.full(D, 2.0**-24),
            np.r_[np.inf, np.ones(D - 1)], np.r_[np.ones(D - 1), -np.inf], np.r_[np.ones(5), np.nan, np.ones(D - 6)],
            np.r_[2.0**-24, np.zeros(D - 1)], np.r_[254.0, np.arange(D - 1) * 2 + 1]]
    if kind == "bf16":
        rows += [rng.standard_normal(D) * 2.0**e for e in (-133, -128, -126, -122, -119, -118, -117, 100, 120)]
    x = np.repeat(np.stack(rows)[:, None], heads, axis=1)
    t, xv = device(x, kind)
    M = len(rows)
    cache = random_cache(2, heads, 32, D, fmt, kind, 10)
    table, pos, entry = np.array([[1]]), np.arange(M), np.zeros(M)
    want = S.write(numpy_of(cache), table, entry, pos, xv, xv[::-1], fmt)
    B.cache_write(cache, ints(table), ints(pos), t, t.flip(0).contiguous(), entry=ints(entry))
    _same(cache, want, f"{fmt} {kind}")
    assert np.isnan(values(cache.k_scale)[1, 0, 11:14]).all()


READS = [(1, 1, 1, 16, 16, 1), (2, 40, 2, 128, 64, 2), (3, 100, 3, 80, 16, 8), (1, 513, 2, 64, 256, 3), (5, 65, 24, 112, 32, 5)]


@pytest.mark.parametrize("shape", READS)
@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_read_against_torch(shape, fmt, kind):
    B_, rows, heads, D, page, T = shape
    rng = np.random.default_rng(sum(shape))
    cache = random_cache(B_ * T, heads, page, D, fmt, kind, 11)
    table = random_table(B_, T, B_ * T, 12)
    if B_ > 2:
        table[1, 0], table[2, -1] = -1, B_ * T
    k, v, there = S.dense(numpy_of(cache), table)
    n = rng.integers(0, T * page + 9, B_)
    n[0] = T * page
    for start in (None, rng.integers(-3, T * page + 3, B_)):
        wide = torch.full((B_, rows + 3, 2 * heads, D + 8), -7.0, dtype=DTYPES[kind], device="cuda")
        ko, vo = wide[:, 2:rows + 2, :heads, :D], wide[:, 2:rows + 2, heads:, :D]
        want = wide.cpu()
        for b in range(B_):
            for j in range(rows):
                p = j + (0 if start is None else int(start[b]))
                if 0 <= p < min(n[b], T * page) and there[b, p]:
                    # the product of a code and an fp32 scale is exact in 64 bits: rounded to fp32, then to the type
                    for at, x in ((slice(0, heads), k), (slice(heads, 2 * heads), v)):
                        want[b, j + 2, at, :D] = torch.from_numpy(x[b, p].astype(np.float32)).to(DTYPES[kind])
        B.cache_read(cache, ints(table), ints(n), ko, vo, start=None if start is None else ints(start))
        torch.cuda.synchronize()
        assert torch.equal(wide.cpu(), want), f"{shape} {fmt} {kind} start {start}"


@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
def test_round_trip(fmt):
    """Written and read back: within half a step of each format (the scale's rounding 2^-24 beside it)."""
    cache = B.KVCache.empty(20, 3, 96, page=32, format="bf16" if fmt == "values" else fmt)
    table = ints(random_table(2, 10, 20, 13))
    k, v = _tokens(500, 3, 96, "bf16", 14)
    entry, pos = ints(np.arange(500) % 2), ints(np.arange(500) // 2)
    B.cache_write(cache, table, pos, k, v, entry=entry)
    back = torch.empty((2, 2, 250, 3, 96), dtype=torch.bfloat16, device="cuda")
    B.cache_read(cache, table, ints([250, 250]), back[0], back[1])
    for x, y in ((k, back[0]), (v, back[1])):
        x, y = values(x), values(y.transpose(0, 1).reshape(500, 3, 96))
        if fmt == "values":
            assert np.array_equal(x, y)
            continue
        top = np.abs(x).max(-1, keepdims=True)
        step = top / 127 / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0**-4, top / 224 * 2.0**-10)
        assert np.all(np.abs(x - y) <= step * (1 + 2.0**-20) + np.abs(y) * 2.0**-8)


def test_pages_far_apart():
    """Pages of a cache that stands beside others in one allocation, past 2^32 bytes."""
    heads, page, D = 2, 16, 64
    far = (1 << 32) + 4096                             # elements from page to page
    room = {n: torch.zeros(2 * far + heads * page * D, dtype=torch.int8, device="cuda") for n in "kv"}
    k = room["k"].as_strided((3, heads, page, D), (far, page * D, D, 1))
    v = room["v"].as_strided((3, heads, D, page), (far, page * D, page, 1))
    sc = torch.zeros((2, 3, 5, heads, page), device="cuda")
    cache = B.KVCache(k, v, sc[0, :, 1], sc[1, :, 1])
    kn, vn = _tokens(40, heads, D, "bf16", 15)
    table, entry, pos = np.array([[2, 0, 1]]), np.zeros(40), np.arange(40)
    want = S.write(numpy_of(cache), table, entry, pos, values(kn), values(vn), "int8")
    B.cache_write(cache, ints(table), ints(pos), kn, vn, entry=ints(entry))
    _same(cache, want, "far")
    ko, vo = torch.empty((2, 1, 40, heads, D), dtype=torch.bfloat16, device="cuda")
    B.cache_read(cache, ints(table), ints([40]), ko, vo)
    dk, dv, _ = S.dense(want, table)
    for got, x in ((ko, dk), (vo, dv)):
        assert torch.equal(got.cpu(), torch.from_numpy(x[:, :40].astype(np.float32)).bfloat16())


def test_another_stream():
    """The call runs on the stream it is given, after what that stream holds."""
    cache = B.KVCache.empty(8, 4, 128, page=64)
    table, pos, entry = ints(np.arange(8)[None]), ints(np.arange(300)), ints(np.zeros(300))
    k, v = _tokens(300, 4, 128, "bf16", 16)
    src = torch.zeros_like(k.contiguous()), torch.zeros_like(v.contiguous())
    out = torch.empty((2, 1, 300, 4, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn((4096, 4096), device="cuda")
    with torch.cuda.stream(side):
        for _ in range(4):
            big = big @ big * 1e-3                     # the stream is busy when the copies are queued
        src[0].copy_(k)
        src[1].copy_(v)
    B.cache_write(cache, table, pos, src[0], src[1], entry=entry, stream=side)
    B.cache_read(cache, table, ints([300]), out[0], out[1], stream=side)
    side.synchronize()
    want = S.write(numpy_of(B.KVCache.empty(8, 4, 128, page=64)), np.arange(8)[None], np.zeros(300), np.arange(300),
                   values(k), values(v), "int8")
    _same(cache, want, "side stream")
    dk = S.dense(want, np.arange(8)[None])[0][:, :300]
    assert torch.equal(out[0].cpu(), torch.from_numpy(dk.astype(np.float32)).bfloat16())
