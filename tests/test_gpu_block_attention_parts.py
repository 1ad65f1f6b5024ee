"""Blocks of 128 rows whose keys are shared by several blocks, with shared
heads and with a padded head dimension: sampled heads against the 64-bit
oracle, in every mode.  Bounds as in tests/test_gpu_block_attention.py."""
import numpy as np
import pytest

import rank_gemm_svdq_amd as B
from tests.block_util import values
from tests.test_gpu_block_attention import _check, _gpu, _make

pytestmark = pytest.mark.gpu


def _arguments(shape, mode):
    B_, Sq, Skv, Hq = shape[:4]
    rng = np.random.default_rng(sum(shape))
    kw = {}
    if mode in ("causal", "cap", "prefix", "everything"):
        kw["causal"] = True
    if mode in ("cap", "everything"):
        kw["softcap"] = 5.0
    if mode in ("slopes", "everything"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq)
    if mode in ("lengths", "everything"):
        kw["kv_len"] = rng.integers(Skv // 4, Skv + 1, B_)
    if mode in ("prefix", "everything"):
        kw["prefix"] = rng.integers(0, Skv + 1, B_)
    if mode in ("documents", "everything"):
        kw["k_doc"] = np.sort(rng.integers(-2, 3, (B_, Skv)), axis=1)
        kw["q_doc"] = rng.integers(-2, 4, (B_, Sq)) if mode == "documents" else kw["k_doc"][:, -Sq:]
    return kw


def _compare(shape, kind, mode, heads):
    B_, Sq, Skv, Hq, Hkv, D = shape
    assert B.attention_workspace_bytes(*shape) > 0
    assert Sq * (Hq // Hkv) > 32 and B_ * Hkv * ((Sq * (Hq // Hkv) + 31) // 32) * Skv > 160 * 1024   # not 32 rows a block
    (q, qv), (k, kv), (v, vv) = _make(*shape, kind, 23)
    kw = _arguments(shape, mode)
    o = _gpu(q, k, v, **kw)
    for h in heads:
        g = h // (Hq // Hkv)
        one = dict(kw)
        if "slopes" in kw:
            one["slopes"] = kw["slopes"][h:h + 1]
        _check(o[:, :, h:h + 1], qv[:, :, h:h + 1], kv[:, :, g:g + 1], vv[:, :, g:g + 1], kind, f"{mode} head {h}", **one)


@pytest.mark.parametrize("mode", ["all", "causal", "cap", "slopes", "lengths", "documents", "prefix", "everything"])
@pytest.mark.parametrize("D,kind", [(128, "bf16"), (104, "fp16"), (64, "fp16")])
def test_shared_heads_in_parts(D, kind, mode):
    _compare((1, 330, 2100, 8, 2, D), kind, mode, (1, 6))


def test_a_chunk_of_two_requests():
    _compare((2, 700, 3001, 16, 4, 128), "bf16", "everything", (10,))


def test_same_bits_again():
    (q, _), (k, _), (v, _) = _make(1, 330, 2100, 8, 2, 128, "bf16", 24)
    first = values(_gpu(q, k, v, causal=True))
    assert all(np.array_equal(first, values(_gpu(q, k, v, causal=True))) for _ in range(3))
