"""Helpers of the block operators' GPU tests: 16-bit values both ways and the
half-ulp of a store."""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def values(t):
    """float64 numpy copy of a device tensor."""
    return t.detach().to("cpu").to(torch.float64).numpy()


def device(a, kind):
    """A device tensor of `kind` from numpy values; returns (tensor, its values in 64 bits)."""
    t = torch.from_numpy(np.asarray(a, np.float32)).to(DTYPES[kind]).cuda()
    return t, values(t)


def half_ulp(y, kind):
    """Largest rounding error of storing values near |y|: half a spacing of
    2^-7 (bf16) or 2^-10 (fp16) of the power of two below, at least half the
    smallest subnormal."""
    bits, tiny = (8, 2.0**-134) if kind == "bf16" else (11, 2.0**-25)
    return np.maximum(np.abs(y) * 2.0**-bits, tiny)


def assert_within(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: {int((~np.isfinite(got)).sum())} values are not finite"
    d = np.abs(got - want)
    if (d > bound).any():
        r = d / np.maximum(bound, 1e-300)
        i = np.unravel_index(np.argmax(r), d.shape)
        raise AssertionError(f"{what}: {int((d > bound).sum())} of {d.size} outside the bound; worst at {i}: "
                             f"got {got[i]!r} want {want[i]!r} off {d[i]:.3e} bound {np.broadcast_to(bound, d.shape)[i]:.3e}")
