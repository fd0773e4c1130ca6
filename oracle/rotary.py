"""Rotary positions and the rotated append to a KV cache in fp64 -- test
infrastructure.

Only tests and ``__graft_entry__.smoke()`` may use this module; the CUDA
library never does.

A row x at position p has its first ``2 * len(inv_freq)`` columns taken as
complex numbers a + ib, pair i being columns (i, i + half) or, interleaved,
(2i, 2i + 1), each multiplied by ``mscale * exp(i * p * inv_freq[i])``; the other
columns are copied.  The inverse multiplies by the conjugate, which is the
transpose of the map, i.e. its gradient.
"""
from __future__ import annotations

import numpy as np

from .attention import _np


def pairs(half, interleaved):
    """Column indices of the two sides of each pair."""
    i = np.arange(half)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + half)


def rope(x, positions, inv_freq, *, mscale=1.0, interleaved=False, inverse=False):
    """``x`` [..., H, d] with its leading axes those of ``positions``."""
    x = np.array(_np(x), copy=True)
    f = _np(inv_freq)
    angle = np.asarray(positions, dtype=np.float64)[..., None, None] * f
    turn = mscale * np.exp((-1j if inverse else 1j) * angle)
    a, b = pairs(len(f), interleaved)
    z = (x[..., a] + 1j * x[..., b]) * turn
    x[..., a], x[..., b] = z.real, z.imag
    return x


def seq_of_rows(n_rows, cu_seqlens):
    """For each packed row (sequence, row in it), (-1, 0) where it is in none."""
    cu = _np(cu_seqlens, np.int64)
    out = []
    for r in range(n_rows):
        hit = [(s, r - int(cu[s])) for s in range(len(cu) - 1) if cu[s] <= r < cu[s + 1]]
        out.append(hit[0] if hit else (-1, 0))
    return out


def kvcache_append(k_new, v_new, k_cache, v_cache, cache_seqlens, *, q=None, cu_seqlens_q=None, block_table=None,
                   positions=None, inv_freq=None, mscale=1.0, interleaved=False):
    """``(q_out, k_cache, v_cache, seqlens)`` after the append.  q_out rows of no
    sequence are NaN (not written)."""
    kc, vc = np.array(_np(k_cache), copy=True), np.array(_np(v_cache), copy=True)
    lens = _np(cache_seqlens, np.int64)
    bt = None if block_table is None else _np(block_table, np.int64)
    page = kc.shape[1]
    k, v = _np(k_new), _np(v_new)
    packed = cu_seqlens_q is not None
    lead = k.shape[:1] if packed else k.shape[:2]
    where = np.empty(lead, dtype=object)
    if packed:
        for r, w in enumerate(seq_of_rows(lead[0], cu_seqlens_q)):
            where[r] = w
        n_new = np.diff(_np(cu_seqlens_q, np.int64))
    else:
        for s in range(lead[0]):
            for i in range(lead[1]):
                where[s, i] = (s, i)
        n_new = np.full(lead[0], lead[1])
    out = None if q is None else np.full(_np(q).shape, np.nan)
    pos_in = None if positions is None else _np(positions, np.int64)
    for at in np.ndindex(*lead):
        s, i = where[at]
        if s < 0:
            continue
        j = int(lens[s]) + i
        p = j if pos_in is None else int(pos_in[at])

        def turned(x):
            return x if inv_freq is None else rope(x, p, inv_freq, mscale=mscale, interleaved=interleaved)
        dst = (s, j) if bt is None else (int(bt[s, j // page]), j % page)
        kc[dst], vc[dst] = turned(k[at]), v[at]
        if q is not None:
            out[at] = turned(_np(q)[at])
    return out, kc, vc, lens + n_new
