"""Helpers of the paged cache's and the gated norms' GPU tests: caches on the
device and as the oracle sees them."""
import numpy as np
import torch

import rank_gemm_svdq_amd as B
from oracle import serving as S
from tests.block_util import DTYPES, values

CODES = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}


def numpy_of(cache):
    """A KVCache as oracle.serving takes it."""
    c = {"k": values(cache.k.float()), "v": values(cache.v.float())}
    if cache.k_scale is not None:
        c["ks"], c["vs"] = values(cache.k_scale), values(cache.v_scale)
    return c


def random_cache(pages, heads, page, D, fmt, kind, seed, gain=1.5, device="cuda"):
    """A KVCache with codes (or values of `kind`) in every place; keys times `gain`."""
    rng = np.random.default_rng(seed)
    k = gain * rng.standard_normal((pages, heads, page, D))
    v = rng.standard_normal((pages, heads, page, D)) * np.exp(rng.normal(0, 1, (pages, heads, page, 1)))
    if fmt == "values":
        t = [torch.from_numpy(x.astype(np.float32)).to(DTYPES[kind]) for x in (k, v)]
        sc = [None, None]
    else:
        enc = [S.encode(x.astype(np.float32), fmt) for x in (k, v)]
        t = [torch.from_numpy(c).to(torch.float32).to(CODES[fmt]) for c, _ in enc]
        sc = [torch.from_numpy(s).to(torch.float32).to(device) for _, s in enc]
    return B.KVCache(t[0].to(device), t[1].transpose(2, 3).contiguous().to(device), *sc)


def random_table(B_, T, pages, seed, shared=False):
    """[B_, T] pages in no order, each at most once unless shared."""
    rng = np.random.default_rng(seed)
    t = rng.integers(0, pages, (B_, T)) if shared else rng.permutation(pages)[:B_ * T].reshape(B_, T)
    return t.astype(np.int32)


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
