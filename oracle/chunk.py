"""Attention of a chunk of new tokens over a KV cache in fp64 -- test
infrastructure.

Only tests and ``__graft_entry__.smoke()`` may use this module; the CUDA
library never does.

Sequence s has ``q_len`` query rows and ``kv_len = seqlens_k[s]`` keys in the
cache, off = kv_len - q_len.  Row i keeps key j when the window rules hold and,
with causal, j <= i + off or j < prefix[s].  Logits are built in the order scale,
soft-cap, distance penalty; a row that keeps no key gives O = 0, LSE = -inf.
"""
from __future__ import annotations

import numpy as np

from .attention import _np, softmax_rows


def kept(q_len, kv_len, *, causal=True, prefix=0, window_left=-1, window_right=-1):
    at = np.arange(q_len)[:, None] + (kv_len - q_len)
    j = np.arange(kv_len)[None, :]
    ok = np.ones((q_len, kv_len), dtype=bool)
    if causal:
        ok &= (j <= at) | (j < prefix)
    if window_left >= 0:
        ok &= j >= at - window_left
    if window_right >= 0:
        ok &= j <= at + window_right
    return ok


def attention_chunk(q, k_cache, v_cache, seqlens_k, *, cu_seqlens_q=None, block_table=None, prefix_lens=None,
                    window_left=-1, window_right=-1, softcap=0.0, scale=None, causal=True, alibi_slopes=None, seqs=None):
    """``(out, lse, mass)``: mass is the same weighted mean of |V| instead of V
    (what the roundings of P are relative to).  Rows of no sequence (or not of
    ``seqs``) are NaN."""
    q = _np(q)
    packed = cu_seqlens_q is not None
    Hq, d = q.shape[-2:]
    scale = 1.0 / np.sqrt(d) if not scale or scale <= 0 else scale
    lens = _np(seqlens_k, np.int64)
    cu = _np(cu_seqlens_q, np.int64) if packed else None
    bt = None if block_table is None else _np(block_table, np.int64)
    kc, vc = k_cache, v_cache
    G = Hq // kc.shape[2]
    out = np.full(q.shape, np.nan)
    mass = np.full(q.shape, np.nan)
    lse = np.full((Hq, q.shape[0]) if packed else (q.shape[0], Hq, q.shape[1]), np.nan)
    for s in range(len(lens)) if seqs is None else seqs:
        rows = slice(int(cu[s]), int(cu[s + 1])) if packed else slice(0, q.shape[1])
        qs = q[rows] if packed else q[s]
        n, L = qs.shape[0], int(lens[s])
        if bt is not None:
            used = bt[s][:-(-L // kc.shape[1])]  # only the sequence's own pages are looked at
            K, V = (_np(c[used]).reshape(-1, *c.shape[2:])[:L] for c in (kc, vc))
        else:
            K, V = _np(kc[s][:L]), _np(vc[s][:L])
        ok = kept(n, L, causal=causal, prefix=0 if prefix_lens is None else int(prefix_lens[s]), window_left=window_left,
                  window_right=window_right)
        dist = np.abs(np.arange(n)[:, None] + (L - n) - np.arange(L)[None, :])
        for h in range(Hq):
            x = scale * (qs[:, h] @ K[:, h // G].T)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if alibi_slopes is not None:
                x = x - float(alibi_slopes[h]) * dist
            p, l = softmax_rows(np.where(ok, x, -np.inf))
            o, m = p @ V[:, h // G], p @ np.abs(V[:, h // G])
            if packed:
                out[rows, h], mass[rows, h], lse[h, rows] = o, m, l
            else:
                out[s, :, h], mass[s, :, h], lse[s, h] = o, m, l
    return out, lse, mass
