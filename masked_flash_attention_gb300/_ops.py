"""Binding of the operators around the KV cache: rotary positions, the rotated
append and the attention of a chunk over the cache (argument marshalling only,
as in ``_lib``).

Outputs and workspaces that a call allocates belong to the stream it runs on
(``stream`` if given, else the current one); tensors of another device than
the current one are refused.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._lib import _DTYPES, FA_ERR_INVALID_ARG, FA_OK, FaError, _ref, fa_rope_scaling, lib

_SCALINGS = {"linear": _lib.FA_ROPE_LINEAR, "ntk": _lib.FA_ROPE_NTK, "blend": _lib.FA_ROPE_BLEND,
             "yarn": _lib.FA_ROPE_YARN}

# These calls are short enough for their host side to count (one token's rotation runs 3 us on the
# device), so the structures of one call are packed into one buffer by one struct call and passed
# as addresses: the prototypes below take plain pointers where _lib's take typed ones.  One call of
# fa_rope with its outputs given took 18.7 us when every structure was built on its own.
_raw = ctypes.CDLL(_lib.LIB_PATH)
_TENSOR = ctypes.sizeof(_lib.fa_tensor)
_OPTS = ctypes.sizeof(_lib.fa_opts)
_LAYOUTS = {}  # number of tensors -> (Struct of one fa_opts and that many fa_tensors, buffer type)
_PAD = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())
_OPTS_FMT = "PPNiiIiPPPP"
assert struct.calcsize("@" + _OPTS_FMT) == _OPTS and _TENSOR % 8 == 0


def _prototype(name, n_tensors, scalars):
    f = getattr(_raw, name)
    f.argtypes = [ctypes.c_void_p] * n_tensors + scalars
    f.restype = ctypes.c_int
    return f


_i32, _f32, _ptr = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
_fa_rope = _prototype("fa_rope", 6, [_f32, _i32, _i32, _ptr])
_fa_kvcache_append = _prototype("fa_kvcache_append", 11, [_f32, _i32, _ptr, _ptr])
_CHUNK_SCALARS = [_i32, _i32, _f32, _f32, _i32, _ptr]
_fa_fwd_chunk = _prototype("fa_fwd_chunk", 9, _CHUNK_SCALARS)
_fa_fwd_chunk_plan = _prototype("fa_fwd_chunk_plan", 9, _CHUNK_SCALARS + [_ptr])

try:  # the raw handle of the current stream, without the Stream object around it
    _current_raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _current_raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _device_of(where, tensors):
    """The current CUDA device, on which every given tensor has to be."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for t in tensors:
        if t is not None and (not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0):
            raise FaError(FA_ERR_INVALID_ARG, f"{where} (tensors must be CUDA tensors on the current device)")
    return dev


class _on_stream:
    """Allocations inside belong to the call's stream, if that is not the current one."""

    def __init__(self, stream, dev):
        self.other = None
        if stream is not None and stream != _current_raw_stream(dev):
            self.other = torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev))

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _workspace(nbytes, device):
    """A workspace whose first 256 bytes (all that needs it) are zero-filled."""
    ws = torch.empty(max(256, int(nbytes)), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _event(e):
    return e.cuda_event if e is not None else 0


def _pack(tensors, dev, stream, workspace=None, max_q=0, max_k=0, debug_flags=0, event_begin=None, event_end=None,
          event_attn_end=None, alibi=None):
    """fa_opts and the fa_tensors of ``tensors`` in one buffer: ``(buffer,
    address of the opts, addresses of the tensors, 0 where None)``.  The buffer
    has to live until the call returns."""
    at, vals, base = [], [], _OPTS
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.nbytes) if workspace is not None else (0, 0)
    vals = [_current_raw_stream(dev) if stream is None else stream, ws_ptr, ws_bytes, max_q or 0, max_k or 0, debug_flags, 0,
            _event(event_begin), _event(event_end), alibi.data_ptr() if alibi is not None else 0, _event(event_attn_end)]
    n = 0
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        shape = t.shape
        nd = len(shape)
        if nd > 4:
            raise ValueError("at most 4 dimensions")
        pad = _PAD[nd]
        # an empty tensor may have no storage: a dummy non-null pointer (never read)
        vals += (t.data_ptr() or 16, _DTYPES.get(t.dtype, 0), nd, *shape, *pad, *t.stride(), *pad)
        at.append(base)
        base += _TENSOR
        n += 1
    try:
        layout, kind = _LAYOUTS[n]
    except KeyError:
        layout, kind = _LAYOUTS[n] = (struct.Struct("@" + _OPTS_FMT + "Qii4q4q" * n), ctypes.c_char * (_OPTS + n * _TENSOR))
    buf = kind()
    layout.pack_into(buf, 0, *vals)
    addr = ctypes.addressof(buf)
    return buf, addr, [x if x is None else addr + x for x in at]


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
    dev = _device_of("fa_rope", (q, k, inv_freq, positions, q_out, k_out))
    if k is None and k_out is not None:
        raise FaError(FA_ERR_INVALID_ARG, "fa_rope (k_out without k)")
    if q_out is None or (k is not None and k_out is None):
        with _on_stream(stream, dev):
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            if k is not None and k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    buf, opts, at = _pack((q, k, q_out, k_out, positions, inv_freq), dev, stream, event_begin=event_begin, event_end=event_end)
    rc = _fa_rope(*at, mscale, 1 if interleaved else 0, 1 if inverse else 0, opts)
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
    dev = _device_of("fa_kvcache_append", (k_new, v_new, k_cache, v_cache, cache_seqlens, q, q_out, cu_seqlens_q,
                                           block_table, positions, inv_freq, seqlens_out, workspace))
    if q is None and q_out is not None:
        raise FaError(FA_ERR_INVALID_ARG, "fa_kvcache_append (q_out without q)")
    with _on_stream(stream, dev):
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if seqlens_out is None:
            seqlens_out = torch.empty_like(cache_seqlens, dtype=torch.int32)
        if workspace is None:
            workspace = _workspace(_lib.FA_KVCACHE_APPEND_WORKSPACE_BYTES, k_new.device)
    buf, opts, at = _pack((q, q_out, k_new, v_new, k_cache, v_cache, cu_seqlens_q, cache_seqlens, block_table, positions,
                           inv_freq, seqlens_out), dev, stream, workspace, event_begin=event_begin, event_end=event_end)
    rc = _fa_kvcache_append(*at[:11], mscale, 1 if interleaved else 0, at[11], opts)
    if rc != FA_OK:
        raise FaError(rc, "fa_kvcache_append")
    return q_out, seqlens_out, workspace


def _lse_shape(q, cu_seqlens_q):
    return (q.shape[1], q.shape[0]) if cu_seqlens_q is not None else (q.shape[0], q.shape[2], q.shape[1])


def fa_fwd_chunk_plan(q, k_cache, v_cache, seqlens_k, *, out=None, lse=None, cu_seqlens_q=None, block_table=None,
                      prefix_lens=None, window_left=-1, window_right=-1, softcap=0.0, scale=None, causal=True,
                      max_seqlen_q=None, max_seqlen_k=None, debug_flags=0, stream=0, **_):
    """Host-only plan query of fa_fwd_chunk; returns (status, plan dict)."""
    if lse is None:
        lse = torch.empty(_lse_shape(q, cu_seqlens_q), dtype=torch.float32, device=q.device)
    buf, opts, at = _pack((q, k_cache, v_cache, q if out is None else out, lse, cu_seqlens_q, seqlens_k, block_table,
                           prefix_lens), -1, stream, max_q=max_seqlen_q, max_k=max_seqlen_k, debug_flags=debug_flags)
    plan = _lib.fa_plan()
    rc = _fa_fwd_chunk_plan(*at, window_left, window_right, softcap, scale or 0.0, 1 if causal else 0, opts,
                            ctypes.addressof(plan))
    return rc, plan.as_dict()


def fa_fwd_chunk(q, k_cache, v_cache, seqlens_k, *, out=None, lse=None, cu_seqlens_q=None, block_table=None,
                 prefix_lens=None, window_left=-1, window_right=-1, softcap=0.0, scale=None, causal=True,
                 max_seqlen_q=None, max_seqlen_k=None, workspace=None, stream=None, debug_flags=0, event_begin=None,
                 event_end=None, event_attn_end=None, alibi_slopes=None):
    """Attention of each sequence's chunk of new tokens over the KV cache
    (fa_fwd_chunk of the C ABI): sequence s sees its first ``seqlens_k[s]``
    cached keys, the chunk's own among them.  ``max_seqlen_k`` is required,
    ``max_seqlen_q`` with ``cu_seqlens_q``.  Returns ``(out, lse, workspace)``,
    allocated with torch when not given; raises FaError on a non-zero status."""
    dev = _device_of("fa_fwd_chunk", (q, k_cache, v_cache, seqlens_k, out, lse, cu_seqlens_q, block_table, prefix_lens,
                                      workspace, alibi_slopes))
    if alibi_slopes is not None:
        alibi_slopes = _lib._alibi(alibi_slopes, q)
    tensors = [q, k_cache, v_cache, out, lse, cu_seqlens_q, seqlens_k, block_table, prefix_lens]
    scalars = (window_left, window_right, softcap, scale or 0.0, 1 if causal else 0)
    if out is None or lse is None or workspace is None:
        with _on_stream(stream, dev):
            if out is None:
                tensors[3] = out = torch.empty_like(q, memory_format=torch.contiguous_format)
            if lse is None:
                tensors[4] = lse = torch.empty(_lse_shape(q, cu_seqlens_q), dtype=torch.float32, device=q.device)
            if workspace is None:
                buf, opts, at = _pack(tensors, dev, stream, max_q=max_seqlen_q, max_k=max_seqlen_k)
                plan = _lib.fa_plan()
                rc = _fa_fwd_chunk_plan(*at, *scalars, opts, ctypes.addressof(plan))
                if rc != FA_OK:
                    raise FaError(rc, "fa_fwd_chunk_plan")
                workspace = _workspace(plan.workspace_bytes, q.device)
    buf, opts, at = _pack(tensors, dev, stream, workspace, max_seqlen_q, max_seqlen_k, debug_flags, event_begin, event_end,
                          event_attn_end, alibi_slopes)
    rc = _fa_fwd_chunk(*at, *scalars, opts)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_chunk")
    return out, lse, workspace
