"""A transformer block's attention half on the package's kernels: residual
sum + RMS norm with FP8 codes, FP8 QKV projection, rotary positions with
several axes (keys straight into the cache), attention over the cache, and the
SVDQuant linear as the output projection.  A prompt first, then one token at
a time.

    python examples/attention_block.py [--tokens 4096] [--steps 8]

Random weights of a FLUX-shaped layer (3072 wide, 24 heads of 128); prints the
time of the prompt and of a token.
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


class AttentionBlock:
    """Weights, rotary plan and K/V cache of one block for one sequence."""

    def __init__(self, width, heads, kv_heads, head_dim, axes, max_len, fmt="mxfp4", rank=32, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.width, self.heads, self.kv_heads, self.head_dim = width, heads, kv_heads, head_dim
        self.norm = (1 + 0.1 * rnd(width)).bfloat16()
        n = (heads + 2 * kv_heads) * head_dim
        self.wqkv, self.sqkv = fp8_blocks(rnd(n, width) / width ** 0.5)
        self.bqkv = (0.1 * rnd(n)).bfloat16()
        self.plan = B.RopePlan(axes, theta=10000.0)
        self.k = torch.zeros((1, max_len, kv_heads, head_dim), dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.used = torch.zeros(1, dtype=torch.int32, device="cuda")   # keys in the cache
        self.len = 0
        inner = heads * head_dim
        w = (S.random_bf16(seed, (inner, width)) / inner ** 0.5).astype(np.float32)
        self.prep = B.prepare(w, np.ones(inner, np.float32), 0.5, rank, fmt)
        self.out = B.DeviceLayer(self.prep)

    def __call__(self, x, positions, residual=None):
        """x, residual [M, width] bf16, positions [M, axes] int32: the next M
        tokens.  Returns (h = x + residual, attention output [M, heads *
        head_dim], projected output [M, width])."""
        M = x.shape[0]
        H, G, D = self.heads, self.kv_heads, self.head_dim
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=x.device)
        h, q, s = new(M, self.width), new(M, self.width, dtype=torch.float8_e4m3fn), \
            new(M, -(-self.width // B.FP8_BLOCK), dtype=torch.float32)
        B.add_rmsnorm_quantize(x, self.norm, 1e-6, q, s, residual=residual, h=h)
        qkv = new(M, (H + 2 * G) * D)
        B.fp8_linear(q, s, self.wqkv, self.sqkv, qkv, bias=self.bqkv)
        qkv = qkv.view(M, H + 2 * G, D)
        place = slice(self.len, self.len + M)
        B.rope(self.plan, positions, qkv[:, :H], qkv[:, :H], qkv[:, H:H + G], self.k[0, place])
        self.v[0, place] = qkv[:, H + G:]
        self.len += M
        self.used.fill_(self.len)
        o = new(1, M, H, D)
        qr = qkv[None, :, :H]
        B.attention(qr, self.k, self.v, o, B.attention_workspace(qr, self.k), causal=True, kv_len=self.used)
        y = new(M, self.width)
        o = o.view(M, H * D)
        B.linear_forward(self.out, o, y, self.out.workspace(M))
        return h, o, y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = AttentionBlock(3072, 24, 24, 128, (16, 56, 56), a.tokens + a.steps + 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def step(M):
        x = torch.randn((M, block.width), generator=g, device="cuda").bfloat16()
        at = torch.arange(block.len, block.len + M, device="cuda")
        pos = torch.stack([at // 4096, at // 64 % 64, at % 64], 1).to(torch.int32)   # 64 x 64 patches an image
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = block(x, pos, residual=x)[2]
        torch.cuda.synchronize()
        return (time.perf_counter() - t) * 1e6, y

    block(torch.zeros((1, block.width), dtype=torch.bfloat16, device="cuda"),
          torch.zeros((1, 3), dtype=torch.int32, device="cuda"))                 # first calls
    block.len = 0
    us, y = step(a.tokens)
    print(f"prompt of {a.tokens} tokens: {us:.0f} us")
    print("tokens after it:", ", ".join(f"{step(1)[0]:.0f}" for _ in range(a.steps)), "us")
    assert bool(torch.isfinite(y.float()).all())


if __name__ == "__main__":
    main()
