"""Queries and keys normalised for each head and rotated, and the gradients, in
fp64 -- test infrastructure.

Only tests and ``__graft_entry__.smoke()`` may use this module; the CUDA
library never does.

y = rope(w * x * r), r = (mean(x^2) + eps)^(-1/2) over the head's columns.  The
gradient is the transpose of the Jacobian J of x -> w x r, which is
J = diag(w) r (I - r^2 x x^T / d), built here as a matrix.
"""
from __future__ import annotations

import numpy as np

from .attention import _np
from .rotary import rope


def norm(x, w=None, eps=1e-6):
    x = _np(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * _np(w)


def norm_rope(x, positions, inv_freq, *, w=None, eps=1e-6, mscale=1.0, interleaved=False):
    """``x`` [..., H, d]; ``inv_freq`` None: no rotation."""
    y = norm(x, w, eps)
    return y if inv_freq is None else rope(y, positions, inv_freq, mscale=mscale, interleaved=interleaved)


def norm_rope_grad(dy, x, positions, inv_freq, *, w=None, eps=1e-6, mscale=1.0, interleaved=False):
    """``(dx, dw)`` for dL/dy = ``dy``."""
    x, g = _np(x), _np(dy)
    d = x.shape[-1]
    if inv_freq is not None:
        g = rope(g, positions, inv_freq, mscale=mscale, interleaved=interleaved, inverse=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).reshape(-1, d).sum(0)
    gw = g if w is None else g * _np(w)
    jac = r[..., None] * (np.eye(d) - (r * r)[..., None] * x[..., :, None] * x[..., None, :] / d)
    return np.einsum("...ij,...j->...i", jac, gw), dw
