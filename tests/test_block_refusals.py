"""More refusals of the block operators' C entries (CPU: every argument is
checked before any device call; the pointers are never followed)."""
import ctypes as C

import numpy as np
import pytest

import rank_gemm_svdq_amd as B

P, Q = 1 << 20, 1 << 24     # aligned addresses
ARG, SHAPE = 1, 2


@pytest.mark.parametrize("change", [dict(h=P, hst=256), dict(h=P, xst=256), dict(h=Q, hst=256, rst=128), dict(h=Q, rst=136)])
def test_norm_in_place_with_another_stride(change):
    a = dict(x=P, xst=128, r=Q, rst=128, w=P, eps=1e-6, M=4, K=128, dtype=0, h=P, hst=128, q=P, s=P)
    a.update(change)
    assert B.lib().svdq_add_rmsnorm_quantize(a["x"], a["xst"], a["r"], a["rst"], a["w"], a["eps"], a["M"], a["K"],
                                             a["dtype"], a["h"], a["hst"], a["q"], a["s"], None) == ARG


@pytest.mark.parametrize("dims,theta", [([16], 1e-300), ([16, 112], 1e-33), ([64], 5e-324)])
def test_frequencies_beyond_fp32(dims, theta):
    """A position below 2^24 times a frequency has to stay finite."""
    with pytest.raises(B.SvdqError) as e:
        B.rope_frequencies(dims, theta)
    assert e.value.status == ARG


def test_the_largest_frequencies_are_finite():
    turns, _ = B.rope_frequencies([16, 112], 1e-31)
    assert np.isfinite(turns).all() and np.isfinite(turns * np.float32((1 << 24) - 1)).all()


@pytest.mark.parametrize("B_,Hq,Sq,status", [(1 << 24, 1, 1, SHAPE), (1 << 10, 1 << 14, 1, SHAPE), (1 << 18, 1, 1 << 13, SHAPE)])
def test_more_attention_heads_than_a_launch_takes(B_, Hq, Sq, status):
    """2^24 blocks of 256 threads are one too many for a grid."""
    from tests.test_oracle_block import _attn_args
    a = _attn_args(B=B_, Hq=Hq, Hkv=Hq, Sq=Sq, Skv=16, D=8)
    assert B.attention_workspace_bytes(B_, Sq, 16, Hq, Hq, 8) == 0
    assert B.lib().svdq_attention(C.byref(a), P, 1 << 40, None) == status
