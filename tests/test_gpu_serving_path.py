"""The serving operators run together as examples/paged_serving.py does.

A request's tokens at once and in pieces (a shorter prompt, then one token at a time)
meet the same cache of codes, and take different kernels for the linear and for
attention.  Q, K and V may differ by one bf16 rounding (2^-8 of a value), which a code of
8 bits answers by at most one step more, and attention's weights by another: for bf16
pages 4 x 2^-8 of the outputs' norm covers both, and codes add a step of
K's and V's largest, 2^-7 for INT8 against values whose root mean square is a
third or less of it, 2^-3 for E4M3 in few elements (2^-8 / 2^-3 of them change)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_gemm_svdq_amd as B
from oracle import serving as S
from tests.block_util import assert_within, half_ulp, values
from tests.gpu_util import rel_fro
from tests.serving_util import ints, numpy_of, random_cache, random_table

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _module():
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _tokens(n, width, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((n, width), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("format", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,D,page", [(8, 2, 64, 16), (4, 1, 128, 64)])
def test_pieces_agree_with_the_whole(format, heads, kv_heads, D, page):
    E = _module()
    width, M, R = 512, 157, 3
    make = lambda: E.PagedBlock(width, heads, kv_heads, D, R, 200, page=page, format=format)
    xs = [_tokens(M, width, s) for s in range(R)]
    whole = make()
    want = [whole.prompt(b, x, x) for b, x in enumerate(xs)]
    piece = make()
    first = (151, 147, 90)
    got = [[piece.prompt(b, x[:n], x[:n])] for b, (x, n) in enumerate(zip(xs, first))]
    for b, more in ((2, 57), (1, 4)):                  # a chunk after a cached start
        n = first[b]
        got[b].append(piece.prompt(b, xs[b][n:n + more], xs[b][n:n + more]))
    assert piece.used.tolist() == [151, 151, 147]
    rest = [x[n:] for x, n in zip(xs, piece.used.tolist())]
    for i in range(6):
        x = torch.stack([r[i] for r in rest])
        out = piece.step(x, x)
        for b in range(R):
            got[b].append([t[b:b + 1] for t in out])
    # request 2 is four tokens behind
    for b in range(R):
        n = 157 if b < 2 else 153
        g, w = ([torch.cat([p[k] for p in got[b]])[:n] for k in range(3)], [t[:n] for t in want[b]])
        assert torch.equal(g[0][:first[b]], w[0][:first[b]])
        tol = {"bf16": 4 * 2.0**-8, "int8": 4 * 2.0**-8 + 3 * 2.0**-7, "fp8": 4 * 2.0**-8 + 2.0**-3 * 2.0**-2.5}[format]
        assert rel_fro(values(g[2]), values(w[2])) <= tol


@pytest.mark.parametrize("format", ["int8", "bf16"])
def test_a_captured_step_replays_as_it_runs(format):
    """Steps from a graph, with eager work between the replays: the same bits as eager steps, the cache's too."""
    E = _module()
    width, R = 256, 4
    make = lambda: E.PagedBlock(width, 4, 2, 64, R, 1600, page=32, format=format, seed=3)
    eager, graphed = make(), make()
    for b in range(R):
        x = _tokens(1500 - 400 * b, width, b)
        for block in (eager, graphed):
            block.prompt(b, x, x)
    x = _tokens(R, width, 9)
    xg = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(xg, xg)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager.step(x, x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graphed.step(xg, xg)
    for i in range(5):
        x = _tokens(R, width, 20 + i)
        xg.copy_(x)
        want = eager.step(x, x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), f"replay {i}"
        assert torch.equal(eager.used, graphed.used)
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in
                   ((eager.cache.k, graphed.cache.k), (eager.cache.v, graphed.cache.v)))
    del g


def test_two_graphs_may_share_a_workspace():
    """Replays in turn, each with parts of its own size."""
    cache = random_cache(200, 2, 64, 64, "int8", "bf16", 1)
    calls = []
    for seed, T, n in ((2, 100, [6400, 5000]), (3, 60, [3840, 33])):
        t = ints(random_table(2, T, 200, seed))
        q = torch.randn((2, 8, 64), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
        calls.append((q, t, ints(n), torch.empty_like(q)))
    ws = B.paged_attention_workspace(calls[0][0], cache, calls[0][1])
    want = []
    for q, t, n, o in calls:
        B.paged_attention(q, cache, t, n, o, ws)
        want.append(o.clone())
    torch.cuda.synchronize()
    graphs = []
    for q, t, n, o in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.paged_attention(q, cache, t, n, o, ws)
        graphs.append(g)
    for i in range(6):
        for g, (_, _, _, o), w in zip(graphs, calls, want):
            o.zero_()
            if i % 2:
                torch.cuda.synchronize()
                ws.fill_(0xFF)                         # what it held before does not matter
            g.replay()
        torch.cuda.synchronize()
        for (_, _, _, o), w in zip(calls, want):
            assert torch.equal(o, w), f"replay {i}"
    del graphs


@pytest.mark.parametrize("fmt", ["int8", "fp8", "values"])
def test_written_then_attended(fmt):
    """Tokens written one step at a time, each attended to by its own query, against the oracle on what the device holds."""
    R, heads, Hq, D, page, T = 3, 2, 6, 80, 16, 4
    kind = "fp16" if fmt == "values" else "bf16"
    dt = torch.float16 if fmt == "values" else torch.bfloat16
    cache = B.KVCache.empty(R * T, heads, D, page=page, format="fp16" if fmt == "values" else fmt)
    table = random_table(R, T, R * T, 5)
    used = torch.tensor([0, 15, 31], dtype=torch.int32, device="cuda")
    host = S.write(numpy_of(cache), table, [], [], [], [], fmt)
    tab, n0 = ints(table), [0, 15, 31]
    k0 = torch.randn((46, heads, D), device="cuda").to(dt)
    e0, p0 = np.r_[np.ones(15), np.full(31, 2)], np.r_[np.arange(15), np.arange(31)]
    B.cache_write(cache, tab, ints(p0), k0, k0, entry=ints(e0))
    host = S.write(host, table, e0, p0, values(k0), values(k0), fmt)
    for i in range(20):
        q, k, v = (torch.randn((R, h, D), device="cuda").to(dt) for h in (Hq, heads, heads))
        B.cache_write(cache, tab, used, k, v)
        host = S.write(host, table, None, np.array(n0) + i, values(k), values(v), fmt)
        used += 1
        o = torch.empty_like(q)
        B.paged_attention(q, cache, tab, used, o, B.paged_attention_workspace(q, cache, tab))
        want, mean, _, _, _ = S.paged_attention(values(q), host, table, np.array(n0) + i + 1, D ** -0.5)
        assert_within(values(o), want, 2.0**-9 * (mean + np.abs(want)) + half_ulp(want, kind), f"step {i}")
    got = numpy_of(cache)
    assert all(np.array_equal(got[n], host[n]) for n in host)
