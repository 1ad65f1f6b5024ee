"""Several requests served by one transformer block: prompts of any length, then
a token of each at a time, keys and values in a paged 8-bit cache.

    norm with FP8 codes -> FP8 QKV projection -> rotary positions -> cache_write
    -> paged_attention (a prompt: cache_read and attention) -> SVDQuant linear
    -> gated_norm: the gated residual sum and the norm of what follows

    python examples/paged_serving.py [--requests 16] [--tokens 2000] [--steps 8]

Random weights of a 4096 wide layer (32 heads of 128 on 8); prints the time of a
prompt and of a step, and of a step replayed from a graph.
"""

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rank_gemm_svdq_amd as B  # noqa: E402
from rank_gemm_svdq_amd import synthetic as S  # noqa: E402


def fp8_blocks(w):
    """E4M3 codes [N, K] and fp32 scales of 128 x 128 blocks of a weight [N, K] (a checkpoint brings these)."""
    N, K = w.shape
    pad = torch.nn.functional.pad(w.float(), (0, 0, 0, -N % B.FP8_BLOCK))
    b = pad.view(-1, B.FP8_BLOCK, K // B.FP8_BLOCK, B.FP8_BLOCK)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / 448.0
    q = (b / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1, K)[:N]
    return q.contiguous(), s.contiguous()


class PagedBlock:
    """Weights of a block and the cache of up to `requests` requests of up to `max_len` tokens."""

    def __init__(self, width, heads, kv_heads, head_dim, requests, max_len, page=64, format="int8", seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.width, self.heads, self.kv_heads, self.head_dim = width, heads, kv_heads, head_dim
        self.norm, self.after, self.next = ((1 + 0.1 * rnd(width)).bfloat16() for _ in range(3))
        self.gate = (0.5 + 0.1 * rnd(1, width)).bfloat16()
        n = (heads + 2 * kv_heads) * head_dim
        self.wqkv, self.sqkv = fp8_blocks(rnd(n, width) / width ** 0.5)
        self.plan = B.RopePlan((head_dim,), theta=10000.0, shared=True, interleaved=False)
        inner = heads * head_dim
        w = (S.random_bf16(seed, (inner, width)) / inner ** 0.5).astype(np.float32)
        self.out = B.DeviceLayer(B.prepare(w, np.ones(inner, np.float32), 0.5, 16, "mxfp4"))
        # every request's pages, handed out in an order of no pattern
        T = -(-max_len // page)
        self.cache = B.KVCache.empty(requests * T, kv_heads, head_dim, page=page, format=format)
        order = torch.randperm(requests * T, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = order.view(requests, T).cuda()
        self.used = torch.zeros(requests, dtype=torch.int32, device="cuda")     # tokens of each request
        self.space = B.paged_attention_workspace(torch.empty((requests, heads, head_dim), device="cuda"), self.cache, self.table)

    def _new(self, *s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="cuda")

    def _qkv(self, x, residual, entry, position):
        """h = x + residual, and the turned queries [M, heads, D]; keys and values go to the cache."""
        M, H, G, D = x.shape[0], self.heads, self.kv_heads, self.head_dim
        h, q, s = self._new(M, self.width), self._new(M, self.width, dtype=torch.float8_e4m3fn), \
            self._new(M, -(-self.width // B.FP8_BLOCK), dtype=torch.float32)
        B.add_rmsnorm_quantize(x, self.norm, 1e-6, q, s, residual=residual, h=h)
        qkv = self._new(M, (H + 2 * G) * D)
        B.fp8_linear(q, s, self.wqkv, self.sqkv, qkv)
        qkv = qkv.view(M, H + 2 * G, D)
        B.rope(self.plan, position.view(M, 1), qkv[:, :H], qkv[:, :H], qkv[:, H:H + G], qkv[:, H:H + G])
        B.cache_write(self.cache, self.table, position, qkv[:, H:H + G], qkv[:, H + G:], entry=entry)
        return h, qkv[:, :H]

    def _end(self, h, o):
        """(h + gate norm(projection), its norm for what follows)"""
        M = h.shape[0]
        p, h2, y = self._new(M, self.width), self._new(M, self.width), self._new(M, self.width)
        B.linear_forward(self.out, o, p, self.out.workspace(M))
        B.gated_norm(p, y=y, h=h2, residual=h, post="rms", post_weight=self.after, gate=self.gate, weight=self.next)
        return h2, y

    def prompt(self, request, x, residual):
        """The next tokens x [M, width] of one request.  Returns (h, y, attention output)."""
        M, start = x.shape[0], int(self.used[request])
        position = torch.arange(start, start + M, dtype=torch.int32, device="cuda")
        h, q = self._qkv(x, residual, torch.full_like(position, request), position)
        self.used[request] += M
        k, v = (self._new(1, start + M, self.kv_heads, self.head_dim) for _ in range(2))
        n = self.used[request:request + 1]
        B.cache_read(self.cache, self.table[request:request + 1], n, k, v)
        o = self._new(1, M, self.heads, self.head_dim)
        B.attention(q[None], k, v, o, B.attention_workspace(q[None], k), causal=True, kv_len=n)
        o = o.view(M, -1)
        return (*self._end(h, o), o)

    def step(self, x, residual):
        """The next token of every request, x [requests, width].  Returns (h, y, attention output).  Launches only, so
        that a graph may hold it."""
        h, q = self._qkv(x, residual, None, self.used)
        self.used += 1
        o = self._new(x.shape[0], self.heads, self.head_dim)
        B.paged_attention(q, self.cache, self.table, self.used, o, self.space)
        o = o.view(x.shape[0], -1)
        return (*self._end(h, o), o)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--tokens", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = PagedBlock(4096, 32, 8, 128, a.requests, a.tokens + 2 * a.steps + 4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda M: torch.randn((M, block.width), generator=g, device="cuda").bfloat16()

    def timed(f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        r = f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) * 1e6, r

    for b in range(a.requests):
        x = rnd(a.tokens)
        us, _ = timed(lambda: block.prompt(b, x, x))
    print(f"prompt of {a.tokens} tokens: {us:.0f} us")
    x = rnd(a.requests)
    print(f"a token of {a.requests} requests:", ", ".join(f"{timed(lambda: block.step(x, x))[0]:.0f}" for _ in range(a.steps)), "us")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, x)[1]
    print("replayed:", ", ".join(f"{timed(graph.replay)[0]:.0f}" for _ in range(a.steps)), "us")
    assert bool(torch.isfinite(y.float()).all())


if __name__ == "__main__":
    main()
