"""Tolerances of fa_qk_norm_rope and its gradients.

r: the sum of d squares in fp32 has no cancellation, its terms go through at most 16
+ 3 roundings, the mean and eps add two, the square root halves them, and the
reciprocal square root is good to 2 ulp (2.4e-7): below 1e-6 relative.  x r w rounds
twice more: NORM = 1.2e-6 relative in each element of the normalised row.
The rotation adds 5e-7 of the pair's magnitude (rope_util).  So y is off by (NORM +
5e-7) mscale (|a| + |b|) plus its own rounding.

Gradients: g = R^T dy carries 5e-7 of its pair's magnitude G = |ga| + |gb| (mscale
included), u = x r 1.2e-6, their products with w 1e-7 each, the mean of d products
21 roundings of 6e-8 over S = mean(G w |u|): dx = r (g w - u mean) is off by
r (2e-6 G w + 6e-6 |u| S) with room for the last two operations.  dw sums g u over N
rows: 2e-6 of each |G u| and, in a chain of at most n additions, n 2^-24 of their
sum; n <= 32 + N / 16 (a lane's share is at least a 32nd of a CTA's rows at d = 128, a
64th at d = 64; one CTA's chain is the longest that any grid makes)."""
import numpy as np
import torch

from oracle import qknorm as N
from oracle.rotary import pairs

NORM = 1.2e-6


def pair_size(x, half, interleaved):
    """|a| + |b| of each element's pair (|x| itself where nothing is rotated)."""
    m = np.abs(x)
    if half:
        a, b = pairs(half, interleaved)
        s = m[..., a] + m[..., b]
        m = m.copy()
        m[..., a] = m[..., b] = s
    return m


def rounding(ref, dtype):
    t = torch.finfo(dtype).eps / 2 * np.abs(ref)
    return t + 2.0 ** -25 if dtype == torch.float16 else t


def within(got, ref, tol, name):
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size}, worst {np.nanmax(np.abs(g - ref)[bad] / tol[bad]):.3g} of the tolerance"


def assert_normed(got, x, pos, f, *, w=None, eps=1e-6, mscale=1.0, interleaved=False, name="y"):
    half = 0 if f is None else len(f)
    ref = N.norm_rope(x, pos, f, w=w, eps=eps, mscale=mscale, interleaved=interleaved)
    mag = pair_size(N.norm(x, w, eps), half, interleaved)
    mag[..., :2 * half] *= abs(mscale)
    within(got, ref, rounding(ref, got.dtype) + (NORM + 5e-7) * 1.01 * mag, name)


def assert_grad(got, dw, dy, x, pos, f, *, w=None, eps=1e-6, mscale=1.0, interleaved=False, name="dx"):
    half = 0 if f is None else len(f)
    ref, rw = N.norm_rope_grad(dy, x, pos, f, w=w, eps=eps, mscale=mscale, interleaved=interleaved)
    x64, g64 = x.double().cpu().numpy(), dy.double().cpu().numpy()
    r = 1.0 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
    G = pair_size(g64, half, interleaved)
    G[..., :2 * half] *= abs(mscale)
    wv = np.ones(x64.shape[-1]) if w is None else np.abs(w.double().cpu().numpy())
    u = np.abs(x64) * r
    S = (G * wv * u).mean(-1, keepdims=True)
    within(got, ref, rounding(ref, got.dtype) + r * (2e-6 * G * wv + 6e-6 * u * S) * 1.01, name)
    if dw is not None:
        n = 32 + x64.size // x64.shape[-1] / 16
        total = (G * u).reshape(-1, x64.shape[-1]).sum(0)
        within(dw, rw, (2e-6 + n * 2.0 ** -24) * total + 2.0 ** -24 * np.abs(rw), name + "'s weight")
