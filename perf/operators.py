"""Workloads of the transformer-block operators that stand beside the quantized linear layer: the residual sum
with root-mean-square norm and 8-bit output, the FP8 linear that reads it, rotary positions with several axes on
the result, and attention.

`run` computes them in elementary torch operations in 32 bits, or with the package's kernels where `own` is true.
The sizes are those of the package's synthetic layers (3072 -> 9216 = Q | K | V in 24 heads of 128, 3072 <-> 12288,
4096 tokens for one image, 8192 for two), cut down, made ragged, and with shared K/V heads and caches beside them.
"""

import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0
BLOCK = 128
EPS = 1e-6
DEV = "cuda"


def _dtype(case):
    return torch.float16 if case["type"] == "fp16" else torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token in flight: the launch is all that counts
        dict(name="norm_token", op="norm", M=1, K=3072, residual=True, type="bf16"),
        # the residual stream of one image ahead of its QKV projection
        dict(name="norm_image", op="norm", M=4096, K=3072, residual=True, type="bf16"),
        # a ragged batch in fp16, last scale block partial, first norm of a block (no residual)
        dict(name="norm_ragged", op="norm", M=1531, K=5000, residual=False, type="fp16"),
        # one token through the QKV projection: the weights are read once for it
        dict(name="linear_token", op="linear", M=1, K=3072, N=9216, bias=True, type="bf16"),
        # a short ragged prompt through the down projection
        dict(name="linear_prompt", op="linear", M=333, K=12288, N=3072, bias=False, type="fp16"),
        # one image through the QKV projection
        dict(name="linear_image", op="linear", M=4096, K=3072, N=9216, bias=True, type="bf16"),
        # a few requests' next tokens, three axes, sixteen lanes of time and the rest for height and width
        dict(name="rope_tokens", op="rope", M=16, Hq=32, Hkv=8, D=128, axes="16,56,56", interleaved=False,
             shared=True, type="fp16"),
        # 512 text tokens and one image of 64 x 64 patches, all heads
        dict(name="rope_image", op="rope", M=4608, Hq=24, Hkv=24, D=128, axes="16,56,56", interleaved=True,
             shared=False, type="bf16"),
        # one new token for each of 16 requests against caches of up to 16384, shared K/V heads, capped scores
        dict(name="attn_token", op="attn", B=16, Sq=1, Skv=16384, Hq=32, Hkv=8, D=128, causal=True, cap=30.0,
             slopes=False, docs=0, prefix=False, ragged=True, type="bf16"),
        # text and one image attending to each other
        dict(name="attn_image", op="attn", B=1, Sq=4608, Skv=4608, Hq=24, Hkv=24, D=128, causal=False, cap=0.0,
             slopes=False, docs=0, prefix=False, ragged=False, type="bf16"),
        # five images of different sizes packed into one row, each seeing itself
        dict(name="attn_packed", op="attn", B=1, Sq=5173, Skv=5173, Hq=24, Hkv=8, D=64, causal=False, cap=0.0,
             slopes=False, docs=5, prefix=False, ragged=False, type="fp16"),
        # a chunk of new tokens after a cached start, a prefix that all see, distance bias
        dict(name="attn_chunk", op="attn", B=2, Sq=700, Skv=3001, Hq=16, Hkv=4, D=128, causal=True, cap=50.0,
             slopes=True, docs=0, prefix=True, ragged=True, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "rope", "attn", "attn"])
    kind = rng.choice(["bf16", "fp16"])
    if op == "norm":
        return dict(op=op, M=_log(rng, 1, 8192), K=8 * _log(rng, 32, 1536), residual=rng.random() < 0.7, type=kind)
    if op == "linear":
        K, N = 128 * _log(rng, 2, 96), 16 * _log(rng, 16, 768)
        return dict(op=op, M=_log(rng, 1, max(2, min(8192, 4096 * 3072 * 9216 // (K * N)))), K=K, N=N,
                    bias=rng.random() < 0.5, type=kind)
    if op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 24])
        Hq = 24 if Hkv == 24 else Hkv * rng.choice([1, 2, 4])
        axes = rng.choice(["16,56,56", "44,42,42", "128", "32,48,48"] if D == 128 else ["16,24,24", "64", "32,32"])
        return dict(op=op, M=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, axes=axes, interleaved=rng.random() < 0.5,
                    shared=rng.random() < 0.5, type=kind)
    D, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    cap, slopes = rng.choice([0.0, 0.0, 30.0, 50.0]), rng.random() < 0.3
    if rng.random() < 0.4:      # new tokens against caches
        B, Skv = rng.randint(1, 16), _log(rng, 17, 16384)
        return dict(op=op, B=B, Sq=rng.choice([1, 1, 1, 2, 5]), Skv=Skv, Hq=Hkv * G, Hkv=Hkv, D=D, causal=True,
                    cap=cap, slopes=slopes, docs=0, prefix=False, ragged=True, type=kind)
    Sq = _log(rng, 8, 4608)
    cached = rng.random() < 0.4
    Skv = Sq + (_log(rng, 1, 2048) if cached else 0)
    causal = cached or rng.random() < 0.5
    B = max(1, min(4, 24 * 4608 * 4608 // (Hkv * G * Sq * Skv)))
    G = max(1, min(G, 24 * 4608 * 4608 // (Hkv * B * Sq * Skv)))
    return dict(op=op, B=B, Sq=Sq, Skv=Skv, Hq=Hkv * G, Hkv=Hkv, D=D, causal=causal, cap=cap, slopes=slopes,
                docs=0 if cached else rng.choice([0, 0, 2, 5]), prefix=causal and rng.random() < 0.4,
                ragged=B > 1 and rng.random() < 0.5, type=kind)


# ------------------------------------------------------------------ inputs

def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _quantized(v, tile):
    """e4m3 codes and fp32 scales of blocks of `tile` rows x 128 columns (the last row block may be partial)."""
    rows, K = v.shape
    pad = -rows % tile
    b = torch.nn.functional.pad(v, (0, 0, 0, pad)).view((rows + pad) // tile, tile, K // BLOCK, BLOCK)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / FP8_MAX
    q = (b / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(rows + pad, K)[:rows].contiguous(), s.contiguous()


def _prepare_norm(case, g, dt):
    M, K = case["M"], case["K"]
    hot = torch.randint(0, K, (max(1, K // 100),), generator=g, device=DEV)     # outlier channels
    x = torch.randn((M, K), generator=g, device=DEV)
    x[:, hot] *= 20.0
    st = {"x": x.to(dt), "w": (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(dt), "r": None}
    if case["residual"]:
        st["r"] = (3.0 * torch.randn((M, K), generator=g, device=DEV)).to(dt)
    st["h"] = torch.empty((M, K), dtype=dt, device=DEV)
    st["q"] = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=DEV)
    st["s"] = torch.empty((M, -(-K // BLOCK)), dtype=torch.float32, device=DEV)
    return st


def _prepare_linear(case, g, dt):
    M, K, N = case["M"], case["K"], case["N"]
    x = torch.randn((M, K), generator=g, device=DEV)
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device=DEV)] *= 20.0
    st = {}
    st["xq"], st["xs"] = _quantized(x, 1)
    st["wq"], st["ws"] = _quantized(torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K), BLOCK)
    st["bias"] = (0.1 * torch.randn((N,), generator=g, device=DEV)).to(dt) if case["bias"] else None
    st["y"] = torch.empty((M, N), dtype=dt, device=DEV)
    return st


def _prepare_rope(case, g, dt):
    M, Hq, Hkv, D = case["M"], case["Hq"], case["Hkv"], case["D"]
    dims = [int(a) for a in case["axes"].split(",")]
    qkv = torch.randn((M, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dt)
    # frame or running token, then the place on a grid of patches
    top = [4096] + [128] * (len(dims) - 1)
    pos = torch.stack([torch.randint(0, t, (M,), generator=g, device=DEV) for t in top], 1).to(torch.int32)
    return {"qkv": qkv, "pos": pos, "dims": dims,
            "qo": torch.empty((M, Hq, D), dtype=dt, device=DEV), "ko": torch.empty((M, Hkv, D), dtype=dt, device=DEV)}


def _prepare_attn(case, g, dt):
    B, Sq, Skv, Hq, Hkv, D = (case[k] for k in ("B", "Sq", "Skv", "Hq", "Hkv", "D"))
    st = {"q": torch.randn((B, Sq, Hq, D), generator=g, device=DEV).mul_(1.5).to(dt),
          "k": torch.randn((B, Skv, Hkv, D), generator=g, device=DEV).mul_(1.5).to(dt),
          "v": torch.randn((B, Skv, Hkv, D), generator=g, device=DEV).to(dt),
          "o": torch.empty((B, Sq, Hq, D), dtype=dt, device=DEV),
          "scale": 1.0 / math.sqrt(D), "len": None, "slopes": None, "prefix": None, "qdoc": None, "kdoc": None}
    if case["ragged"]:
        lo = max(Sq, Skv // 4)
        st["len"] = torch.randint(lo, Skv + 1, (B,), generator=g, device=DEV).to(torch.int32)
    if case["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
    if case["prefix"]:
        st["prefix"] = torch.randint(0, max(1, Skv // 3) + 1, (B,), generator=g, device=DEV).to(torch.int32)
    if case["docs"]:
        ends = torch.sort(torch.randint(0, Skv, (B, case["docs"] - 1), generator=g, device=DEV), dim=1).values
        at = torch.arange(Skv, device=DEV)
        doc = (at[None, :, None] >= ends[:, None, :]).sum(-1).to(torch.int32)
        st["kdoc"] = doc.contiguous()
        st["qdoc"] = doc[:, Skv - Sq:].contiguous()
    return st


def prepare(case, seed):
    make = {"norm": _prepare_norm, "linear": _prepare_linear, "rope": _prepare_rope, "attn": _prepare_attn}
    st = make[case["op"]](case, _rng(seed), _dtype(case))
    st["case"] = dict(case)
    return st


# ------------------------------------------------------------- plain forms

def _plain_norm(st):
    x = st["x"].float()
    h = x if st["r"] is None else x + st["r"].float()
    M, K = h.shape
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    y = torch.nn.functional.pad(y, (0, -K % BLOCK)).view(M, -1, BLOCK)
    s = y.abs().amax(-1) / FP8_MAX
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    q = (y * inv[..., None]).to(torch.float8_e4m3fn).view(M, -1)[:, :K].contiguous()
    return {"h": h.to(st["x"].dtype), "q": q, "s": s}


def _plain_linear(st):
    N, K = st["wq"].shape
    x = (st["xq"].float().view(-1, K // BLOCK, BLOCK) * st["xs"][..., None]).view(-1, K)
    ws = st["ws"].repeat_interleave(BLOCK, 0)[:N]
    w = (st["wq"].float().view(N, K // BLOCK, BLOCK) * ws[..., None]).view(N, K)
    y = x @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(st["y"].dtype)


def _plain_rope(st):
    case = st["case"]
    dims, Hq, Hkv = st["dims"], case["Hq"], case["Hkv"]
    dev = st["qkv"].device
    if case["shared"]:      # one ladder of frequencies through all axes
        f = torch.pow(10000.0, -torch.arange(0, sum(dims), 2, device=dev).float() / sum(dims))
    else:                   # a ladder for each axis
        f = torch.cat([torch.pow(10000.0, -torch.arange(0, d, 2, device=dev).float() / d) for d in dims])
    p = torch.cat([st["pos"][:, a:a + 1].expand(-1, d // 2) for a, d in enumerate(dims)], 1).float()
    c, s = torch.cos(p * f)[:, None, :], torch.sin(p * f)[:, None, :]
    x = st["qkv"][:, :Hq + Hkv].float()
    half = x.shape[-1] // 2
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    y = y.to(st["qkv"].dtype)
    return {"q": y[:, :Hq].contiguous(), "k": y[:, Hq:].contiguous()}


def _plain_attn(st):
    case = st["case"]
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    dev = q.device
    n = st["len"].long() if st["len"] is not None else torch.full((B,), Skv, device=dev)
    pos = (n - Sq)[:, None] + torch.arange(Sq, device=dev)                    # [B, Sq]
    key = torch.arange(Skv, device=dev)
    see = (key[None, None, :] < n[:, None, None]).expand(B, Sq, Skv)
    if case["causal"]:
        past = key[None, None, :] <= pos[:, :, None]
        if st["prefix"] is not None:
            past = past | (key[None, None, :] < st["prefix"].long()[:, None, None])
        see = see & past
    if st["qdoc"] is not None:
        see = see & (st["qdoc"][:, :, None] == st["kdoc"][:, None, :])
    qg = q.view(B, Sq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B * Hkv, G * Sq, D)
    kt = k.permute(0, 2, 3, 1).reshape(B * Hkv, D, Skv).contiguous()
    s = torch.bmm(qg, kt).mul_(st["scale"]).view(B, Hkv, G, Sq, Skv)
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    if st["slopes"] is not None:
        far = (pos[:, :, None] - key[None, None, :]).abs().float()
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    t = s.sum(-1, keepdim=True)
    o = torch.bmm(s.view(B * Hkv, G * Sq, Skv), v.permute(0, 2, 1, 3).reshape(B * Hkv, Skv, D).contiguous())
    o = o.view(B, Hkv, G, Sq, D) / torch.where(t > 0, t, torch.ones_like(t))
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(st["q"].dtype)


# ------------------------------------------------------ the package's calls

def _own_norm(st):
    import rank_gemm_svdq_amd as B
    B.add_rmsnorm_quantize(st["x"], st["w"], EPS, st["q"], st["s"], residual=st["r"], h=st["h"])
    return {"h": st["h"], "q": st["q"], "s": st["s"]}


def _own_linear(st):
    import rank_gemm_svdq_amd as B
    B.fp8_linear(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], bias=st["bias"])
    return st["y"]


def _own_rope(st):
    import rank_gemm_svdq_amd as B
    case = st["case"]
    if "plan" not in st:        # frequencies of a model: made once, kept by the program
        st["plan"] = B.RopePlan(st["dims"], theta=10000.0, shared=case["shared"], interleaved=case["interleaved"])
    Hq, Hkv = case["Hq"], case["Hkv"]
    B.rope(st["plan"], st["pos"], st["qkv"][:, :Hq], st["qo"], st["qkv"][:, Hq:Hq + Hkv], st["ko"])
    return {"q": st["qo"], "k": st["ko"]}


def _own_attn(st):
    import rank_gemm_svdq_amd as B
    case = st["case"]
    if "space" not in st:       # kept by the program between calls
        st["space"] = B.attention_workspace(st["q"], st["k"])
    B.attention(st["q"], st["k"], st["v"], st["o"], st["space"], scale=st["scale"], causal=case["causal"],
                softcap=case["cap"], slopes=st["slopes"], kv_len=st["len"], prefix=st["prefix"], q_doc=st["qdoc"],
                k_doc=st["kdoc"])
    return st["o"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "rope": _plain_rope, "attn": _plain_attn}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        n = M * K
        return {"bytes": n * 2 * (2 + case["residual"]) + n + 2 * K + 4 * M * -(-K // BLOCK), "flops": 8 * n}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        kb = K // BLOCK
        return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // BLOCK)) + 2 * M * N + 2 * N * case["bias"],
                "flops": 2 * M * N * K}
    if case["op"] == "rope":
        n = case["M"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 4 * n + 4 * case["M"] * len(case["axes"].split(",")), "flops": 3 * n}
    B, Sq, Skv, Hq, Hkv, D = (case[k] for k in ("B", "Sq", "Skv", "Hq", "Hkv", "D"))
    keys = Skv * (0.625 if case["ragged"] else 1.0)             # lengths are uniform over the upper three quarters
    seen = Sq * keys
    if case["causal"] and Sq > 1:
        seen = Sq * (keys - Sq / 2.0)
        if case["prefix"]:                                      # a sixth of the cache on average
            seen = max(seen, Sq * Skv / 6.0)
    if case["docs"]:
        seen *= 2.0 / (case["docs"] + 1)                        # expected share of pairs with uniform cuts
    return {"bytes": 2.0 * B * D * (2 * Sq * Hq + 2 * keys * Hkv), "flops": 4.0 * B * Hq * D * max(seen, Sq)}


# ------------------------------------------------------------------- exact

def _exact_norm(case, st):
    h = st["x"].double()
    if st["r"] is not None:
        h = h + st["r"].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + EPS) * st["w"].double()
    q, s = torch.empty_like(y), torch.empty(st["s"].shape, dtype=torch.float64, device=DEV)
    for b in range(s.shape[1]):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = part.abs().max(1).values / FP8_MAX
        q[:, b * BLOCK:(b + 1) * BLOCK] = part / s[:, b:b + 1]
    return {"h": h, "q": q, "s": s}


def _exact_linear(case, st):
    y = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device=DEV)
    col = torch.arange(case["N"], device=DEV) // BLOCK
    for b in range(case["K"] // BLOCK):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        wt = st["wq"][:, at].double().t().contiguous()
        y += (st["xq"][:, at].double() @ wt) * st["xs"][:, b].double()[:, None] * st["ws"][:, b].double()[col]
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_rope(case, st):
    x = st["qkv"][:, :case["Hq"] + case["Hkv"]].double()
    y = x.clone()
    half, j = x.shape[-1] // 2, 0
    for a, d in enumerate(st["dims"]):
        for i in range(d // 2):
            f = 10000.0 ** (-2.0 * j / sum(st["dims"])) if case["shared"] else 10000.0 ** (-2.0 * i / d)
            t = (st["pos"][:, a].double() * f)[:, None]
            u, v = (2 * j, 2 * j + 1) if case["interleaved"] else (j, half + j)
            y[..., u] = x[..., u] * torch.cos(t) - x[..., v] * torch.sin(t)
            y[..., v] = x[..., u] * torch.sin(t) + x[..., v] * torch.cos(t)
            j += 1
    return {"q": y[:, :case["Hq"]].contiguous(), "k": y[:, case["Hq"]:].contiguous()}


def _exact_attn(case, st):
    B, Sq, Skv, Hq, Hkv, D = (case[k] for k in ("B", "Sq", "Skv", "Hq", "Hkv", "D"))
    out = torch.zeros((B, Sq, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(st["len"][b]) if st["len"] is not None else Skv
        place = torch.arange(n - Sq, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        hidden = torch.zeros((Sq, n), dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= j > place
            if st["prefix"] is not None:
                hidden &= j >= int(st["prefix"][b])
        if st["kdoc"] is not None:
            hidden |= st["qdoc"][b][:, None] != st["kdoc"][b][None, :n]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            z = st["q"][b, :, h].double() @ st["k"][b, :n, g].double().t().contiguous() * st["scale"]
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * (place - j).abs()
            z[hidden] = -math.inf
            p = torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
            out[b, :, h] = p @ st["v"][b, :n, g].double().contiguous()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    f = {"norm": _exact_norm, "linear": _exact_linear, "rope": _exact_rope, "attn": _exact_attn}[case["op"]]
    v = f(case, st)
    return {k: x.cpu().numpy().astype(np.float64) for k, x in v.items()} if isinstance(v, dict) else v.cpu().numpy()
