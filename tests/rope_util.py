"""Tolerance of the rotary operators, shared by their tests.

A rotated element is m (a c - b s) in fp32 (or with the sides swapped).  The
angle's fraction of a turn is cut to 32 bits and rounded to fp32: at most
2^-31 + 2^-25 half turns, 9.6e-8 rad.  sincospif is good to 2 ulp (2^-23 near 1,
1.2e-7 each, taken twice for the two factors' sum), m times it rounds by 2^-24,
the two products and their sum by 2^-24 each.  Together each of a, b carries less
than 9.6e-8 + 1.2e-7 + 4 * 6e-8 < 5e-7 of its magnitude times m.  The result is
then rounded once to its type: half a step, eps / 2 of the value (fp16 also half
its smallest subnormal, 2^-25)."""
import numpy as np
import torch


def assert_rotated(got, ref, x, inv_freq, mscale, interleaved, name=""):
    """``got`` (a 16-bit torch tensor) against the fp64 rotation ``ref`` of ``x``."""
    from oracle.rotary import pairs
    half = len(inv_freq)
    eps = torch.finfo(got.dtype).eps / 2
    mag = np.zeros(ref.shape)
    a, b = pairs(half, interleaved)
    xs = np.abs(x.double().cpu().numpy()) if isinstance(x, torch.Tensor) else np.abs(x)
    mag[..., a] = mag[..., b] = xs[..., a] + xs[..., b]
    f32 = 5e-7 * abs(mscale) * mag
    tol = eps * np.abs(ref) + f32 * (1 + eps)
    tol[..., 2 * half:] = 0.0  # copied
    if got.dtype == torch.float16:
        tol[..., :2 * half] += 2.0 ** -25
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size}, worst {np.nanmax(np.abs(g - ref)[bad])}"
