"""Binding of the operators around attention: rotary positions and the
rotated append to a KV cache (argument marshalling only, as in ``_lib``).

Outputs and workspaces that a call allocates belong to the stream it runs on
(``stream`` if given, else the current one); tensors of another device than
the current one are refused.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import FA_ERR_INVALID_ARG, FA_OK, FaError, _ref, describe, fa_rope_scaling, lib, make_opts

_SCALINGS = {"linear": _lib.FA_ROPE_LINEAR, "ntk": _lib.FA_ROPE_NTK, "blend": _lib.FA_ROPE_BLEND,
             "yarn": _lib.FA_ROPE_YARN}


def _check_cuda(where, *tensors):
    """Every given tensor lives on the current CUDA device."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise FaError(FA_ERR_INVALID_ARG, f"{where} (tensors must be CUDA tensors)")
        if dev is None:
            dev = torch.cuda.current_device()
        if t.device.index != dev:
            raise FaError(FA_ERR_INVALID_ARG, f"{where} (tensors must be on the current device, cuda:{dev})")


def _allocating_on(stream, device):
    """Allocations inside belong to ``stream`` (a raw handle; None: the current stream)."""
    if stream is None or stream == torch.cuda.current_stream(device).cuda_stream:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device))


def _workspace(nbytes, device):
    """A workspace whose first 256 bytes (all that needs it) are zero-filled."""
    ws = torch.empty(max(256, int(nbytes)), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _set_workspace(opts, workspace):
    opts.workspace = workspace.data_ptr()
    opts.workspace_bytes = workspace.numel() * workspace.element_size()


def fa_rope_inv_freq(rot, base=10000.0, *, scaling=None, factor=1.0, original_len=0, low=1.0, high=4.0):
    """The ``rot / 2`` rotary frequencies (radians per position) for ``base``
    and their ``mscale``, as ``(fp64 CPU tensor, float)``.  ``scaling``: None,
    "linear", "ntk", "blend" (kept above ``high`` turns in ``original_len``
    positions, divided by ``factor`` below ``low``, mixed between) or "yarn"
    (the same, mixed along the pair index; its usual bounds are low=1,
    high=32).  Host only; raises FaError on arguments that make no sense."""
    if scaling is not None and scaling not in _SCALINGS:
        raise FaError(FA_ERR_INVALID_ARG, f"fa_rope_inv_freq (scaling {scaling!r})")
    sc = None
    if scaling is not None:
        sc = fa_rope_scaling(_SCALINGS[scaling], int(original_len), float(factor), float(low), float(high))
    out = (ctypes.c_double * max(1, int(rot) // 2))()
    m = ctypes.c_float(1.0)
    rc = lib.fa_rope_inv_freq(int(rot), float(base), _ref(sc), out, ctypes.byref(m))
    if rc != FA_OK:
        raise FaError(rc, "fa_rope_inv_freq")
    return torch.tensor(list(out), dtype=torch.float64), m.value


def fa_rope(q, k=None, *, inv_freq, positions=None, q_out=None, k_out=None, mscale=1.0, interleaved=False,
            inverse=False, stream=None, event_begin=None, event_end=None):
    """Rotary positions on ``q`` (and ``k``) through the C ABI; ``inverse`` is
    the backward pass (gradients of the rotated rows in, of the rows out).
    ``inv_freq``: fp64 CUDA tensor [rot/2]; ``positions``: int32 [B, S] or
    [total], optional for [B, S, H, d].  Returns ``(q_out, k_out)``, allocated
    with torch when not given (k_out is None without k).  Raises FaError on a
    non-zero status."""
    _check_cuda("fa_rope", q, k, inv_freq, positions, q_out, k_out)
    if k is None and k_out is not None:
        raise FaError(FA_ERR_INVALID_ARG, "fa_rope (k_out without k)")
    with _allocating_on(stream, q.device):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    opts = make_opts(stream=stream, event_begin=event_begin, event_end=event_end)
    descs = [describe(x) for x in (q, k, q_out, k_out, positions, inv_freq)]
    rc = lib.fa_rope(*[_ref(x) for x in descs], float(mscale), int(bool(interleaved)), int(bool(inverse)),
                     ctypes.byref(opts))
    if rc != FA_OK:
        raise FaError(rc, "fa_rope")
    return q_out, k_out


def fa_kvcache_append(k_new, v_new, k_cache, v_cache, cache_seqlens, *, q=None, q_out=None, cu_seqlens_q=None,
                      block_table=None, positions=None, inv_freq=None, mscale=1.0, interleaved=False,
                      seqlens_out=None, workspace=None, stream=None, event_begin=None, event_end=None):
    """Append the step's keys (rotated when ``inv_freq`` is given) and values
    to the cache, and rotate ``q`` beside them, through the C ABI.  Returns
    ``(q_out, seqlens_out, workspace)``: q_out (None without q), the int32
    lengths after the append, and the workspace holding the error word; each is
    allocated with torch when not given.  Raises FaError on a non-zero status."""
    _check_cuda("fa_kvcache_append", k_new, v_new, k_cache, v_cache, cache_seqlens, q, q_out, cu_seqlens_q,
                block_table, positions, inv_freq, seqlens_out, workspace)
    if q is None and q_out is not None:
        raise FaError(FA_ERR_INVALID_ARG, "fa_kvcache_append (q_out without q)")
    with _allocating_on(stream, k_new.device):
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if seqlens_out is None:
            seqlens_out = torch.empty(cache_seqlens.shape, dtype=torch.int32, device=k_new.device)
        if workspace is None:
            workspace = _workspace(_lib.FA_KVCACHE_APPEND_WORKSPACE_BYTES, k_new.device)
    opts = make_opts(stream=stream, event_begin=event_begin, event_end=event_end)
    _set_workspace(opts, workspace)
    descs = [describe(x) for x in (q, q_out, k_new, v_new, k_cache, v_cache, cu_seqlens_q, cache_seqlens,
                                   block_table, positions, inv_freq)]
    lens = describe(seqlens_out)
    rc = lib.fa_kvcache_append(*[_ref(x) for x in descs], float(mscale), int(bool(interleaved)), _ref(lens),
                               ctypes.byref(opts))
    if rc != FA_OK:
        raise FaError(rc, "fa_kvcache_append")
    return q_out, seqlens_out, workspace
