"""The KV cache held in 8 bits, in fp64 -- test infrastructure.

Only tests and ``__graft_entry__.smoke()`` may use this module; the CUDA
library never does.

An element is ``code * scale``: an e4m3 code (sign, 4 exponent bits with bias 7,
3 mantissa bits; largest 448, no infinities, 0x7f and 0xff NaN) and, for each
block of tokens and head, a power of two 2^E, -40 <= E <= 40: the smallest whose
448-fold holds the block's finite elements.
"""
from __future__ import annotations

import numpy as np

from .attention import _np, softmax_rows
from .rotary import rope, seq_of_rows
from .qknorm import norm

LOW, HIGH = -40, 40


def code_values():
    """The value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7f) == 0x7f, np.nan, v)
    return np.where(c >= 128, -v, v)


_VALUES = code_values()
_POSITIVE = _VALUES[:127]  # 0 .. 448, increasing


def to_code(x):
    """The nearest code's value (ties to the even code), saturated; NaN and infinities give NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    up = (a - _POSITIVE[lo] > _POSITIVE[hi] - a) | ((a - _POSITIVE[lo] == _POSITIVE[hi] - a) & (hi % 2 == 0))
    y = np.where(up, _POSITIVE[hi], _POSITIVE[lo])
    return np.where(np.isfinite(x), np.copysign(y, x), np.nan)


def exponent(top):
    """The block exponent for a largest magnitude ``top``."""
    for e in range(LOW, HIGH + 1):
        if top <= 448.0 * 2.0 ** e:
            return e
    return HIGH


def values(cache):
    """A torch.float8_e4m3fn tensor as fp64, by the codes' bits."""
    import torch
    return _VALUES[cache.view(torch.uint8).cpu().numpy()]


def dequantised(cache, scale):
    """Code values [.., rows, H, d] (fp64) times scales [.., rows / block, H]."""
    s = _np(scale)
    return cache * np.repeat(s, cache.shape[-3] // s.shape[-2], axis=-2)[..., None]


def append(k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens, *, q=None, cu_seqlens_q=None,
           block_table=None, positions=None, inv_freq=None, mscale=1.0, interleaved=False, q_weight=None, k_weight=None,
           eps=None):
    """``k_cache`` and ``v_cache`` as fp64 code values.  Returns a dict: q_out (NaN
    where not written), the code values and scales of both caches after the append, the
    lengths, and ``k_exact`` / ``v_exact``: what the codes of the rows written or
    rounded again stand for before their rounding, over the new scale (NaN elsewhere)."""
    lens = _np(cache_seqlens, np.int64)
    bt = None if block_table is None else _np(block_table, np.int64)
    page = k_cache.shape[1]
    packed = cu_seqlens_q is not None
    x = {"k": _np(k_new), "v": _np(v_new)}
    lead = x["k"].shape[:1] if packed else x["k"].shape[:2]
    if packed:
        where = seq_of_rows(lead[0], cu_seqlens_q)
        n_new = np.diff(_np(cu_seqlens_q, np.int64))
    else:
        where = [(s, i) for s in range(lead[0]) for i in range(lead[1])]
        n_new = np.full(lead[0], lead[1])

    def turned(row, w, j, at):
        y = row if not eps else norm(row, w, eps)
        if inv_freq is None:
            return y
        p = j if positions is None else int(_np(positions, np.int64)[at])
        return rope(y, p, inv_freq, mscale=mscale, interleaved=interleaved)

    out = None if q is None else np.full(_np(q).shape, np.nan)
    res = {"lens": lens + n_new}
    for name, cache, scale in (("k", k_cache, k_scale), ("v", v_cache, v_scale)):
        codes, sc = np.array(cache), np.array(_np(scale))
        block = page // sc.shape[1]
        exact = np.full(codes.shape, np.nan)
        blocks = {}
        for at, (s, i) in zip(np.ndindex(*lead), where):
            if s < 0:
                continue
            j = int(lens[s]) + i
            row = turned(x[name][at], k_weight, j, at) if name == "k" else x[name][at]
            if name == "k" and q is not None:
                out[at] = turned(_np(q)[at], q_weight, j, at)
            blocks.setdefault((s, j // block), []).append((j, row))
        for (s, b), rows in blocks.items():
            j0 = b * block
            pg, r0 = (s, j0) if bt is None else (int(bt[s, j0 // page]), j0 % page)
            bi = r0 // block
            n_old = rows[0][0] - j0
            for h in range(codes.shape[2]):
                a = np.abs(np.stack([r[h] for _, r in rows]))
                e = exponent(a[np.isfinite(a)].max(initial=0.0))
                before = sc[pg, bi, h]
                if n_old and 2.0 ** e <= before:
                    after = before
                else:
                    after = 2.0 ** e
                    if n_old:
                        old = codes[pg, r0:r0 + n_old, h] * (before / after)
                        exact[pg, r0:r0 + n_old, h] = old
                        codes[pg, r0:r0 + n_old, h] = to_code(old)
                sc[pg, bi, h] = after
                for j, r in rows:
                    y = np.where(np.isfinite(r[h]), r[h], np.nan) / after
                    exact[pg, r0 + j - j0, h] = y
                    codes[pg, r0 + j - j0, h] = to_code(y)
        res.update({name: codes, name + "_scale": sc, name + "_exact": exact})
    res["q"] = out
    return res


def kept(q_len, kv_len, *, causal=True, prefix=0, window_left=-1, window_right=-1, sinks=0):
    at = np.arange(q_len)[:, None] + (kv_len - q_len)
    j = np.arange(kv_len)[None, :]
    ok = np.ones((q_len, kv_len), dtype=bool)
    if causal:
        ok &= (j <= at) | (j < prefix)
    if window_left >= 0:
        ok &= (j >= at - window_left) | (j < sinks)
    if window_right >= 0:
        ok &= j <= at + window_right
    return ok


def attention_chunk(q, k, v, seqlens_k, *, cu_seqlens_q=None, block_table=None, prefix_lens=None, sink_keys=0,
                    window_left=-1, window_right=-1, softcap=0.0, scale=None, causal=True, alibi_slopes=None):
    """Over dequantised caches ``k`` and ``v`` (fp64).  ``(out, lse, mass, size)``: mass
    is the weighted mean of |V|, size the largest scale * sum |q k| that a row sees
    (what the logits' rounding errors are relative to).  A kept key whose V is NaN
    makes its column NaN; hidden ones do not matter."""
    q = _np(q)
    packed = cu_seqlens_q is not None
    Hq, d = q.shape[-2:]
    scale = 1.0 / np.sqrt(d) if not scale or scale <= 0 else scale
    lens = _np(seqlens_k, np.int64)
    cu = _np(cu_seqlens_q, np.int64) if packed else None
    bt = None if block_table is None else _np(block_table, np.int64)
    G = Hq // k.shape[2]
    out, mass = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((Hq, q.shape[0]) if packed else (q.shape[0], Hq, q.shape[1]), np.nan)
    size = np.zeros_like(lse)
    for s in range(len(lens)):
        rows = slice(int(cu[s]), int(cu[s + 1])) if packed else slice(0, q.shape[1])
        qs = q[rows] if packed else q[s]
        n, L = qs.shape[0], int(lens[s])
        if bt is not None:
            used = bt[s][:-(-L // k.shape[1])]
            K, V = (c[used].reshape(-1, *c.shape[2:])[:L] for c in (k, v))
        else:
            K, V = k[s][:L], v[s][:L]
        ok = kept(n, L, causal=causal, prefix=0 if prefix_lens is None else int(prefix_lens[s]), window_left=window_left,
                  window_right=window_right, sinks=sink_keys)
        dist = np.abs(np.arange(n)[:, None] + (L - n) - np.arange(L)[None, :])
        for h in range(Hq):
            x = scale * (qs[:, h] @ K[:, h // G].T)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if alibi_slopes is not None:
                x = x - float(alibi_slopes[h]) * dist
            p, l = softmax_rows(np.where(ok, x, -np.inf))
            vh = V[:, h // G]
            nan = np.isnan(vh)
            clean = np.where(nan, 0.0, vh)
            o, m = p @ clean, p @ np.abs(clean)
            o = np.where((ok.astype(float) @ nan) > 0, np.nan, o)
            z = np.where(ok, scale * (np.abs(qs[:, h]) @ np.abs(K[:, h // G]).T), 0.0).max(-1, initial=0.0)
            if packed:
                out[rows, h], mass[rows, h], lse[h, rows], size[h, rows] = o, m, l, z
            else:
                out[s, :, h], mass[s, :, h], lse[s, h], size[s, h] = o, m, l, z
    return out, lse, mass, size
