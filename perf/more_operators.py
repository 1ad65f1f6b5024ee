"""Workloads of the operators of a serving step that stand beside attention and the norms: writing keys and values
into a paged cache in 8 bits (or as they are), reading them back, attention of one new token of each request over the
pages, and the end of a block: norms on both sides of its gate and residual scale.

`run` computes them in elementary torch operations in 32 bits, or with the package's kernels where `own` is true.

A cache: k [pages, heads, page, D] and v [pages, heads, D, page] (values side by side for each element of a head), 16-bit
values or codes, and for codes fp32 scales [pages, heads, page].  `table` [requests, n] names the pages of a request in
the order of its positions.  Codes are x / s rounded to the nearest, with for each token and head
    int8  s = max |x| / 127,        fp8 (E4M3)  s = the least power of two with max |x| / s <= 448.
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
        # the next tokens of 16 requests go into the cache
        dict(name="write_tokens", op="write", B=16, M=16, Hkv=8, D=128, page=64, format="int8", pad=0, type="bf16"),
        # keys and values of 512 text tokens and one image of 64 x 64 patches
        dict(name="write_image", op="write", B=1, M=4608, Hkv=24, D=128, page=64, format="fp8", pad=0, type="bf16"),
        # prompts of five requests in a padded batch, stored as they are in small pages
        dict(name="write_ragged", op="write", B=5, M=1531, Hkv=4, D=64, page=16, format="values", pad=130, type="fp16"),
        # the image's keys and values back, for the prompt that attends to it
        dict(name="read_image", op="read", B=1, S=4608, Hkv=24, D=128, page=64, format="fp8", type="bf16"),
        # parts of five requests' caches ahead of a chunk of new tokens
        dict(name="read_ragged", op="read", B=5, S=3001, Hkv=8, D=64, page=32, format="int8", type="fp16"),
        # one short request: the launches count
        dict(name="paged_token", op="paged", B=1, S=600, Hq=32, Hkv=8, D=128, page=64, format="int8", cap=0.0, window=0,
             slopes=False, type="bf16"),
        # one new token for each of 16 requests against caches of up to 16384 keys
        dict(name="paged_batch", op="paged", B=16, S=16384, Hq=32, Hkv=8, D=128, page=64, format="int8", cap=0.0,
             window=0, slopes=False, type="bf16"),
        # one request with a long document
        dict(name="paged_long", op="paged", B=1, S=131072, Hq=32, Hkv=8, D=128, page=128, format="fp8", cap=30.0,
             window=0, slopes=False, type="bf16"),
        # 40 requests, a head of keys for each of queries, 16-bit pages, the nearest 1500 keys with a distance bias
        dict(name="paged_near", op="paged", B=40, S=3001, Hq=24, Hkv=24, D=64, page=16, format="values", cap=0.0,
             window=1500, slopes=True, type="fp16"),
        # one token between two blocks, normed on both sides
        dict(name="gated_token", op="gated", M=1, E=1, K=4096, post="rms", pre="rms", alpha=1.0, modulate=False,
             codes=False, type="bf16"),
        # text and image of two entries with gate, scale and shift of their own, codes for the next FP8 linear
        dict(name="gated_image", op="gated", M=4608, E=2, K=4096, post="none", pre="layer", alpha=1.0, modulate=True,
             codes=True, type="bf16"),
        # a ragged batch of seven entries in fp16, scaled residual, last scale block partial
        dict(name="gated_ragged", op="gated", M=1531, E=7, K=5000, post="rms", pre="layer", alpha=0.8, modulate=True,
             codes=False, type="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "paged", "paged", "gated"])
    kind, fmt, page = rng.choice(["bf16", "fp16"]), rng.choice(["int8", "fp8", "values"]), rng.choice([16, 32, 64, 128, 256])
    D, Hkv = rng.choice([64, 80, 96, 128]), rng.choice([1, 2, 3, 4, 8, 24])
    if op == "write":
        B = rng.randint(1, 16)
        M = rng.choice([B, _log(rng, B, 4608)])
        return dict(op=op, B=B, M=M, Hkv=Hkv, D=D, page=page, format=fmt, pad=rng.choice([0, 0, M // 9]), type=kind)
    if op == "read":
        S = _log(rng, 16, 4608)
        B = max(1, min(rng.randint(1, 8), 4608 * 24 * 128 // (S * Hkv * D)))
        return dict(op=op, B=B, S=S, Hkv=Hkv, D=D, page=page, format=fmt, type=kind)
    if op == "paged":
        S, G = _log(rng, 1, 65536), rng.choice([1, 2, 4, 5, 8, 16])
        cost = Hkv * D * (2 if fmt == "values" else 1) * max(1, G // 4)
        S = min(S, 16 * 16384 * 8 * 128 // cost)
        B = max(1, min(_log(rng, 1, 64), 16 * 16384 * 8 * 128 // (S * cost)))
        return dict(op=op, B=B, S=S, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, format=fmt, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), slopes=rng.random() < 0.3, type=kind)
    K, E = 8 * _log(rng, 32, 1024), rng.choice([1, 1, 2, 7])
    return dict(op=op, M=_log(rng, 1, min(8192, 4608 * 4096 // K)), E=E, K=K, post=rng.choice(["none", "rms", "layer"]),
                pre=rng.choice(["rms", "layer"]), alpha=rng.choice([1.0, 1.0, 0.8]), modulate=rng.random() < 0.6,
                codes=rng.random() < 0.5, type=kind)


# ------------------------------------------------------------------ inputs

def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _encoded(x, fmt):
    """Codes and scales of the last dimension's vectors."""
    top = x.abs().amax(-1)
    if fmt == "int8":
        s = top / 127.0
        c = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None])     # borders in 64 bits
        return c.to(torch.int8), s
    m, e = torch.frexp(top / FP8_MAX)
    s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), torch.where(m == 0.5, e - 1, e)), torch.zeros_like(top))
    return (x / torch.where(s > 0, s, torch.ones_like(s))[..., None]).to(torch.float8_e4m3fn), s


def _code_type(case):
    return {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "values": _dtype(case)}[case["format"]]


def _table(case, lengths, g, count=None):
    """Pages of each request (-1 where it has none) in an order without a pattern, and how many pages there are."""
    page, need = case["page"], [-(-int(n) // case["page"]) for n in lengths]
    count, width = count or sum(need) + 3, max(need)
    order = torch.randperm(count, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, count


def _lengths(B, lo, hi, seed):
    return [int(n) for n in np.random.RandomState(seed % (1 << 32)).randint(lo, hi + 1, B)]


def _keys(shape, dt, g):
    """Keys have a few channels that stand out."""
    x = torch.randn(shape, generator=g, device=DEV)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=g, device=DEV)
    x[..., hot] *= 6.0
    return x.to(dt)


def _filled(case, pages, g, dt):
    """A cache of `pages` pages with something in every place."""
    Hkv, P, D = case["Hkv"], case["page"], case["D"]
    k = _keys((pages, Hkv, P, D), dt, g)
    v = torch.randn((pages, Hkv, P, D), generator=g, device=DEV).to(dt)
    if case["format"] == "values":
        return {"k": k, "v": v.transpose(2, 3).contiguous(), "ks": None, "vs": None}
    k, ks = _encoded(k.float(), case["format"])
    v, vs = _encoded(v.float(), case["format"])
    return {"k": k, "v": v.transpose(2, 3).contiguous(), "ks": ks, "vs": vs}


def _prepare_write(case, seed, g, dt):
    B, M, Hkv, P, D = (case[k] for k in ("B", "M", "Hkv", "page", "D"))
    # tokens of each request, and where its cache ends so far
    cuts = sorted(_lengths(B - 1, 0, M - B, seed)) if B > 1 else []
    n = [b - a + 1 for a, b in zip([0] + cuts, cuts + [M - B])]
    start = _lengths(B, 0, 3 * P, seed + 1)
    table, pages = _table(case, [s + t for s, t in zip(start, n)], g, M // P + 4 * B + 3)
    entry = np.repeat(np.arange(B), n)
    pos = np.concatenate([np.arange(s, s + t) for s, t in zip(start, n)])
    pos = np.concatenate([pos, np.full(case["pad"], -1)])        # padded rows behind the last request
    entry = np.concatenate([entry, np.zeros(case["pad"], np.int64)])
    qkv = torch.empty((M + case["pad"], 3 * Hkv, D), dtype=dt, device=DEV)      # columns of a QKV output
    qkv[:, Hkv:2 * Hkv] = _keys((M + case["pad"], Hkv, D), dt, g)
    qkv[:, 2 * Hkv:] = torch.randn((M + case["pad"], Hkv, D), generator=g, device=DEV).to(dt)
    st = {"kn": qkv[:, Hkv:2 * Hkv], "vn": qkv[:, 2 * Hkv:], "table": table,
          "entry": torch.tensor(entry, dtype=torch.int32, device=DEV), "pos": torch.tensor(pos, dtype=torch.int32, device=DEV)}
    ct = _code_type(case)
    st["k"] = torch.zeros((pages, Hkv, P, D), dtype=ct, device=DEV)
    st["v"] = torch.zeros((pages, Hkv, D, P), dtype=ct, device=DEV)
    scaled = case["format"] != "values"
    st["ks"] = torch.zeros((pages, Hkv, P), device=DEV) if scaled else None
    st["vs"] = torch.zeros((pages, Hkv, P), device=DEV) if scaled else None
    return st


def _prepare_read(case, seed, g, dt):
    B, S, Hkv, D = (case[k] for k in ("B", "S", "Hkv", "D"))
    # positions start .. start + S of a request, as far as it goes
    n = _lengths(B, max(1, S // 2), S, seed) if B > 1 else [S]
    start = _lengths(B, 0, 2 * case["page"], seed + 1) if B > 1 else [0]
    table, pages = _table(case, [s + t for s, t in zip(start, n)], g)
    st = _filled(case, pages, g, dt)
    st["table"] = table
    st["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    st["len"] = torch.tensor([s + t for s, t in zip(start, n)], dtype=torch.int32, device=DEV)
    st["ko"] = torch.zeros((B, S, Hkv, D), dtype=dt, device=DEV)
    st["vo"] = torch.zeros((B, S, Hkv, D), dtype=dt, device=DEV)
    return st


def _prepare_paged(case, seed, g, dt):
    B, S, Hq, D = (case[k] for k in ("B", "S", "Hq", "D"))
    n = _lengths(B, max(1, S // 4), S, seed) if B > 1 else [S]
    table, pages = _table(case, n, g)
    st = _filled(case, pages, g, dt)
    st["table"] = table
    st["len"] = torch.tensor(n, dtype=torch.int32, device=DEV)
    st["q"] = torch.randn((B, Hq, D), generator=g, device=DEV).mul_(0.8).to(dt)
    st["o"] = torch.empty((B, Hq, D), dtype=dt, device=DEV)
    st["scale"] = 1.0 / math.sqrt(D)
    st["slopes"] = None
    if case["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
    return st


def _prepare_gated(case, seed, g, dt):
    M, E, K = case["M"], case["E"], case["K"]
    x = torch.randn((M, K), generator=g, device=DEV)
    r = 3.0 * torch.randn((M, K), generator=g, device=DEV)
    r[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device=DEV)] *= 20.0      # outlier channels
    st = {"x": x.to(dt), "r": r.to(dt), "post_w": None, "w": None, "mod": None, "entry": None}
    if case["post"] != "none":
        st["post_w"] = (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(dt)
    if case["pre"] == "rms":
        st["w"] = (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(dt)
    if case["modulate"]:        # an entry's gate, scale and shift side by side, as one projection gives them
        st["mod"] = (0.3 * torch.randn((E, 3 * K), generator=g, device=DEV)).to(dt)
        st["entry"] = torch.sort(torch.randint(0, E, (M,), generator=g, device=DEV)).values.to(torch.int32)
    st["h"] = torch.empty((M, K), dtype=dt, device=DEV)
    st["y"] = None if case["codes"] else torch.empty((M, K), dtype=dt, device=DEV)
    st["qc"] = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=DEV) if case["codes"] else None
    st["sc"] = torch.empty((M, -(-K // BLOCK)), device=DEV) if case["codes"] else None
    return st


def prepare(case, seed):
    make = {"write": _prepare_write, "read": _prepare_read, "paged": _prepare_paged, "gated": _prepare_gated}
    st = make[case["op"]](case, seed, _rng(seed), _dtype(case))
    st["case"] = dict(case)
    return st


# ------------------------------------------------------------- plain forms

def _plain_write(st):
    case, P = st["case"], st["case"]["page"]
    live = torch.nonzero(st["pos"] >= 0)[:, 0]
    pos, entry = st["pos"][live].long(), st["entry"][live].long()
    page, at = st["table"][entry, pos // P].long(), pos % P
    for new, codes, scales, turned in ((st["kn"], st["k"], st["ks"], False), (st["vn"], st["v"], st["vs"], True)):
        x = new[live]
        if scales is not None:
            x, s = _encoded(x.float(), case["format"])
            scales[page, :, at] = s
            x, codes = x.view(torch.uint8), codes.view(torch.uint8)
        (codes.transpose(2, 3) if turned else codes)[page, :, at] = x
    return {"k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}


def _pages(codes, scales, table):
    """fp32 values [B, heads, positions, D] of the pages of a table; codes [pages, heads, page, D]."""
    t = table.long().clamp_min(0)
    x = codes[t].float() if scales is None else codes.view(torch.uint8)[t].view(codes.dtype).float()
    if scales is not None:
        x = x * scales[t][..., None]
    B, T, H, P, D = x.shape
    return x.transpose(1, 2).reshape(B, H, T * P, D)


def _plain_read(st):
    S = st["ko"].shape[1]
    at = st["start"].long()[:, None] + torch.arange(S, device=DEV)              # [B, S]
    live = (at < st["len"][:, None])[..., None, None]
    out = {}
    for name, codes, scales, o in (("k", st["k"], st["ks"], st["ko"]), ("v", st["v"].transpose(2, 3), st["vs"], st["vo"])):
        x = _pages(codes, scales, st["table"]).transpose(1, 2)                  # [B, positions, heads, D]
        x = torch.take_along_dim(x, at.clamp_max(x.shape[1] - 1)[..., None, None], dim=1)
        out[name] = torch.where(live, x.to(o.dtype), o)
    return out


def _plain_paged(st):
    case = st["case"]
    B, Hq, D = st["q"].shape
    Hkv, n = case["Hkv"], st["len"].long()[:, None]
    G = Hq // Hkv
    k = _pages(st["k"], st["ks"], st["table"])
    v = _pages(st["v"].transpose(2, 3), st["vs"], st["table"])
    N = k.shape[2]
    j = torch.arange(N, device=DEV)[None]
    see = j < n
    if case["window"]:
        see = see & (j >= n - case["window"])
    q = st["q"].float().view(B * Hkv, G, D)
    s = torch.bmm(q, k.view(B * Hkv, N, D).transpose(1, 2).contiguous()).mul_(st["scale"]).view(B, Hkv, G, N)
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1) * (n - 1 - j).float().abs()[:, None, None]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    t = s.sum(-1, keepdim=True)
    o = torch.bmm(s.view(B * Hkv, G, N), v.view(B * Hkv, N, D)).view(B, Hkv, G, D)
    return (o / torch.where(t > 0, t, torch.ones_like(t))).view(B, Hq, D).to(st["q"].dtype)


def _norm(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x if kind == "none" else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_gated(st):
    case, K = st["case"], st["case"]["K"]
    b = _norm(st["x"].float(), case["post"])
    if st["post_w"] is not None:
        b = b * st["post_w"].float()
    if st["mod"] is not None:
        gate, scale, shift = st["mod"][st["entry"].long()].float().chunk(3, 1)
        b = gate * b
    h = case["alpha"] * st["r"].float() + b
    y = _norm(h, case["pre"])
    if st["w"] is not None:
        y = y * st["w"].float()
    if st["mod"] is not None:
        y = y * (1.0 + scale) + shift
    h = h.to(st["h"].dtype)
    if not case["codes"]:
        return {"h": h, "y": y.to(st["y"].dtype)}
    y = torch.nn.functional.pad(y, (0, -K % BLOCK)).view(y.shape[0], -1, BLOCK)
    s = y.abs().amax(-1) / FP8_MAX
    q = (y / torch.where(s > 0, s, torch.ones_like(s))[..., None]).to(torch.float8_e4m3fn)
    return {"h": h, "q": q.view(h.shape[0], -1)[:, :K].contiguous(), "s": s}


# ------------------------------------------------------ the package's calls

def _cache(st):
    import rank_gemm_svdq_amd as B
    if "cache" not in st:       # kept by the program for the life of the cache
        st["cache"] = B.KVCache(st["k"], st["v"], st["ks"], st["vs"])
    return st["cache"]


def _own_write(st):
    import rank_gemm_svdq_amd as B
    B.cache_write(_cache(st), st["table"], st["pos"], st["kn"], st["vn"], entry=st["entry"])
    return {"k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}


def _own_read(st):
    import rank_gemm_svdq_amd as B
    B.cache_read(_cache(st), st["table"], st["len"], st["ko"], st["vo"], start=st["start"])
    return {"k": st["ko"], "v": st["vo"]}


def _own_paged(st):
    import rank_gemm_svdq_amd as B
    case, cache = st["case"], _cache(st)
    if "space" not in st:       # kept by the program between calls
        st["space"] = B.paged_attention_workspace(st["q"], cache, st["table"])
    B.paged_attention(st["q"], cache, st["table"], st["len"], st["o"], st["space"], scale=st["scale"],
                      softcap=case["cap"], window=case["window"], slopes=st["slopes"])
    return st["o"]


def _own_gated(st):
    import rank_gemm_svdq_amd as B
    case, K, mod = st["case"], st["case"]["K"], st["mod"]
    gate, scale, shift = (None, None, None) if mod is None else (mod[:, :K], mod[:, K:2 * K], mod[:, 2 * K:])
    B.gated_norm(st["x"], y=st["y"], q=st["qc"], s=st["sc"], h=st["h"], residual=st["r"], residual_scale=case["alpha"],
                 post=case["post"], post_weight=st["post_w"], gate=gate, pre=case["pre"], weight=st["w"], scale=scale,
                 shift=shift, entry=st["entry"], eps=EPS)
    return {"h": st["h"], "q": st["qc"], "s": st["sc"]} if case["codes"] else {"h": st["h"], "y": st["y"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "paged": _own_paged, "gated": _own_gated}[op](state)
    return {"write": _plain_write, "read": _plain_read, "paged": _plain_paged, "gated": _plain_gated}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "gated":
        n, M, K = case["M"] * case["K"], case["M"], case["K"]
        small = 2 * K * ((case["post"] != "none") + (case["pre"] == "rms") + 3 * case["E"] * case["modulate"])
        out = n + 4 * M * -(-K // BLOCK) if case["codes"] else 2 * n
        return {"bytes": 6 * n + out + small, "flops": 14 * n}
    Hkv, D = case["Hkv"], case["D"]
    scaled = case["format"] != "values"
    row = Hkv * (2 * D * (1 if scaled else 2) + 8 * scaled)     # of a token in the cache, keys and values
    if case["op"] == "write":
        return {"bytes": case["M"] * (4 * Hkv * D + row) + 8 * (case["M"] + case["pad"]), "flops": 6 * case["M"] * Hkv * D}
    if case["op"] == "read":
        n = case["B"] * case["S"] * (0.75 if case["B"] > 1 else 1.0)            # lengths are uniform over the upper half
        return {"bytes": n * (4 * Hkv * D + row), "flops": 2 * n * Hkv * D}
    B, S, Hq = case["B"], case["S"], case["Hq"]
    keys = S * (0.625 if B > 1 else 1.0)                        # over the upper three quarters
    if case["window"]:
        keys = min(keys, case["window"])
    return {"bytes": B * (keys * row + 4 * Hq * D), "flops": 4.0 * B * Hq * D * max(keys, 1.0)}


# ------------------------------------------------------------------- exact

def _exact_codes(x, fmt):
    """(codes, scales) of vectors along the last axis, scales held in fp32."""
    top = np.abs(x).max(-1)
    if fmt == "int8":
        s = (top / 127.0).astype(np.float32).astype(np.float64)
        return np.rint(x / np.where(s > 0, s, 1.0)[..., None]), s
    s = np.where(top > 0, 2.0 ** np.ceil(np.log2(np.where(top > 0, top, 1.0) / FP8_MAX)), 0.0)
    u = x / np.where(s > 0, s, 1.0)[..., None]
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -20))), -6) - 3)
    return np.rint(u / step) * step, s


def _exact_write(case, st):
    table, entry, pos = (st[k].cpu().numpy() for k in ("table", "entry", "pos"))
    P, out = case["page"], {}
    at = [(m, table[entry[m], pos[m] // P], pos[m] % P) for m in range(len(pos)) if pos[m] >= 0]
    m, page, place = (np.array(c) for c in zip(*at))
    for name, new in (("k", st["kn"]), ("v", st["vn"])):
        x = new.double().cpu().numpy()[m]
        codes = np.zeros((st["k"].shape[0], case["Hkv"], P, case["D"]))
        if case["format"] != "values":
            x, s = _exact_codes(x, case["format"])
            scales = np.zeros(codes.shape[:3])
            scales[page, :, place] = s
            out[name + "s"] = scales
        codes[page, :, place] = x
        out[name] = codes if name == "k" else np.ascontiguousarray(codes.transpose(0, 1, 3, 2))
    if case["format"] == "int8":
        out["k"], out["v"] = out["k"].astype(np.int8), out["v"].astype(np.int8)
    return {k: out.get(k) for k in ("k", "v", "ks", "vs")}


def _exact_keys(st, name, b, lo, n):
    """Values [heads, n - lo, D] at positions lo .. n of request b."""
    codes, scales = st[name], st[name + "s"]
    P = codes.shape[2] if name == "k" else codes.shape[3]
    t = st["table"][b, lo // P:-(-n // P)].long()
    x = (codes if scales is None else codes.view(torch.uint8))[t].view(codes.dtype).double()
    x = x if name == "k" else x.transpose(2, 3)
    if scales is not None:
        x = x * scales[t].double()[..., None]
    x = x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])
    return x[:, lo % P:lo % P + n - lo]


def _exact_read(case, st):
    out = {}
    for name in ("k", "v"):
        o = torch.zeros(st["ko"].shape, dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            lo, n = int(st["start"][b]), int(st["len"][b])
            o[b, :n - lo] = _exact_keys(st, name, b, lo, n).transpose(0, 1)
        out[name] = o.cpu().numpy()
    return out


def _exact_paged(case, st):
    B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(st["len"][b])
        lo = max(0, n - case["window"]) if case["window"] else 0
        k, v = _exact_keys(st, "k", b, lo, n), _exact_keys(st, "v", b, lo, n)
        away = n - 1 - torch.arange(lo, n, device=DEV).double()
        for h in range(Hq):
            g = h // (Hq // Hkv)
            z = (k[g] * st["q"][b, h].double()).sum(1) * st["scale"]
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * away
            out[b, h] = (torch.softmax(z, 0)[:, None] * v[g]).sum(0)
    return out.cpu().numpy()


def _exact_norm(x, kind):
    if kind == "layer":
        x = x - x.sum(1, keepdim=True) / x.shape[1]
    return x if kind == "none" else x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS)


def _exact_gated(case, st):
    K = case["K"]
    b = _exact_norm(st["x"].double(), case["post"])
    if st["post_w"] is not None:
        b *= st["post_w"].double()
    e = st["entry"].long() if st["entry"] is not None else None
    if e is not None:
        b = b * st["mod"][e, :K].double()
    h = case["alpha"] * st["r"].double() + b
    y = _exact_norm(h, case["pre"])
    if st["w"] is not None:
        y = y * st["w"].double()
    if e is not None:
        y = y + y * st["mod"][e, K:2 * K].double() + st["mod"][e, 2 * K:].double()
    if not case["codes"]:
        return {"h": h.cpu().numpy(), "y": y.cpu().numpy()}
    s = torch.stack([y[:, i:i + BLOCK].abs().max(1).values for i in range(0, K, BLOCK)], 1) / FP8_MAX
    q = y / s.repeat_interleave(BLOCK, 1)[:, :K]
    return {"h": h.cpu().numpy(), "q": q.cpu().numpy(), "s": s.cpu().numpy()}


def exact(case, seed):
    st = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "paged": _exact_paged, "gated": _exact_gated}[case["op"]](case, st)
