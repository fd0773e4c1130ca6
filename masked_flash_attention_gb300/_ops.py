"""The operators around the KV cache: norms and rotary positions of queries and
keys, the rotated append and the attention of a chunk over the cache, in the
model's type or in 8 bits.  These calls are short, so their
arguments are marshalled by the compiled module ``_binding``
(``csrc/binding.cpp``); the functions here hold the signatures and raise.

Outputs and workspaces that a call allocates belong to the stream it runs on
(``stream``, a raw handle, if given, else the current one).  Every tensor has
to be a CUDA tensor of the current device: others are refused.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import FA_ERR_INVALID_ARG, FA_OK, FaError, _ref, fa_rope_scaling, lib


class _Unusable:
    """Stands in for a compiled module that is missing or built for something
    else: a call that needs it raises, and the rest of the package works."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{_BINDING} {self._why}: build it with `python -c 'import __graft_entry__ as g; g.build()'`")


_BINDING = _lib.LIB_PATH.replace("libmfa_gb300.so", "_binding.so")
try:
    from . import _binding
except ImportError as e:
    _binding = _Unusable(f"is missing or does not load ({e})")
else:
    _built_for = tuple(getattr(_binding, name, None) for name in ("ABI_VERSION", "TORCH_VERSION"))
    if _built_for != (_lib.ABI_VERSION, torch.__version__):
        _binding = _Unusable("was built for ABI {} and torch {}, ".format(*_built_for) +
                             f"this is ABI {_lib.ABI_VERSION} and torch {torch.__version__}")

_SCALINGS = {"linear": _lib.FA_ROPE_LINEAR, "ntk": _lib.FA_ROPE_NTK, "blend": _lib.FA_ROPE_BLEND,
             "yarn": _lib.FA_ROPE_YARN}


def _event(e):
    return None if e is None else e.cuda_event


def _raise(status, where):
    hint = " (or a tensor that is not on the current CUDA device)" if status == FA_ERR_INVALID_ARG else ""
    raise FaError(status, where + hint)


def fa_rope_inv_freq(rot, base=10000.0, *, scaling=None, factor=1.0, original_len=0, low=1.0, high=4.0):
    """The ``rot / 2`` rotary frequencies (radians per position) for ``base``
    and their ``mscale``, as ``(fp64 CPU tensor, float)``.  ``scaling``: None,
    "linear", "ntk", "blend" (kept above ``high`` turns in ``original_len``
    positions, divided by ``factor`` below ``low``, mixed between) or "yarn"
    (the same, mixed along the pair index; its usual bounds are low=1,
    high=32).  Host only; raises FaError on arguments that make no sense."""
    if scaling is not None and scaling not in _SCALINGS:
        raise FaError(FA_ERR_INVALID_ARG, f"fa_rope_inv_freq (scaling {scaling!r})")
    rot, original_len = int(rot), int(original_len)
    if not (-2**31 <= rot < 2**31 and -2**31 <= original_len < 2**31):  # (ctypes would wrap them)
        raise FaError(FA_ERR_INVALID_ARG, "fa_rope_inv_freq")
    sc = None
    if scaling is not None:
        sc = fa_rope_scaling(_SCALINGS[scaling], original_len, float(factor), float(low), float(high))
    out = (ctypes.c_double * max(1, rot // 2))()
    m = ctypes.c_float(1.0)
    rc = lib.fa_rope_inv_freq(rot, float(base), _ref(sc), out, ctypes.byref(m))
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
    r = _binding.rope(q, k, q_out, k_out, positions, inv_freq, mscale, interleaved, inverse, stream,
                      _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_rope")
    return r[:2]


def fa_kvcache_append(k_new, v_new, k_cache, v_cache, cache_seqlens, *, q=None, q_out=None, cu_seqlens_q=None,
                      block_table=None, positions=None, inv_freq=None, mscale=1.0, interleaved=False,
                      seqlens_out=None, workspace=None, stream=None, event_begin=None, event_end=None):
    """Append the step's keys (rotated when ``inv_freq`` is given) and values
    to the cache, and rotate ``q`` beside them, through the C ABI.  Returns
    ``(q_out, seqlens_out, workspace)``: q_out (None without q), the int32
    lengths after the append, and the workspace holding the error word; each is
    allocated with torch when not given.  Raises FaError on a non-zero status."""
    r = _binding.kvcache_append(k_new, v_new, k_cache, v_cache, cache_seqlens, q, q_out, cu_seqlens_q, block_table,
                                positions, inv_freq, mscale, interleaved, seqlens_out, workspace, stream,
                                _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_kvcache_append")
    return r


def fa_fwd_chunk_plan(q, k_cache, v_cache, seqlens_k, *, out=None, lse=None, cu_seqlens_q=None, block_table=None,
                      prefix_lens=None, window_left=-1, window_right=-1, softcap=0.0, scale=None, causal=True,
                      max_seqlen_q=None, max_seqlen_k=None, debug_flags=0, **_):
    """Host-only plan query of fa_fwd_chunk; returns (status, plan dict)."""
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]) if cu_seqlens_q is not None else (q.shape[0], q.shape[2], q.shape[1]),
                          dtype=torch.float32, device=q.device)
    plan = _lib.fa_plan()
    rc = _binding.fwd_chunk_plan(q, k_cache, v_cache, q if out is None else out, lse, cu_seqlens_q, seqlens_k, block_table,
                                 prefix_lens, window_left, window_right, softcap, scale, causal, max_seqlen_q, max_seqlen_k,
                                 debug_flags, ctypes.addressof(plan))
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
    r = _binding.fwd_chunk(q, k_cache, v_cache, out, lse, cu_seqlens_q, seqlens_k, block_table, prefix_lens, window_left,
                           window_right, softcap, scale, causal, max_seqlen_q, max_seqlen_k, debug_flags, stream, workspace,
                           alibi_slopes, _event(event_begin), _event(event_attn_end), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_fwd_chunk")
    return r


def fa_qk_norm_rope(q, k=None, *, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None, positions=None, q_out=None,
                    k_out=None, mscale=1.0, interleaved=False, stream=None, event_begin=None, event_end=None):
    """``q`` (and ``k``) normalised for each head by its root mean square,
    weighted and rotated, in one pass (fa_qk_norm_rope of the C ABI).  Weights
    are [d], fp32 or q's type, None for ones; without ``inv_freq`` nothing is
    rotated.  Returns ``(q_out, k_out)``, allocated with torch when not given
    (k_out is None without k).  Raises FaError on a non-zero status."""
    r = _binding.qk_norm_rope(q, k, q_weight, k_weight, q_out, k_out, positions, inv_freq, eps, mscale, interleaved, stream,
                              _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_qk_norm_rope")
    return r[:2]


def fa_qk_norm_rope_bwd(dq_out, dk_out, q, k=None, *, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                        positions=None, dq=None, dk=None, dq_weight=None, dk_weight=None, mscale=1.0, interleaved=False,
                        workspace=None, stream=None, event_begin=None, event_end=None):
    """Gradients of fa_qk_norm_rope for the same arguments, from ``dq_out`` and
    ``dk_out`` (None without k).  Returns ``(dq, dk, dq_weight, dk_weight,
    workspace)``, allocated with torch when not given; a weight's gradient (fp32
    [d]) is computed when the weight or a tensor for it is given, else None, and
    the workspace is None where none is needed.  Raises FaError on a non-zero
    status."""
    r = _binding.qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, dq_weight, dk_weight, positions, inv_freq,
                                  eps, mscale, interleaved, workspace, stream, _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_qk_norm_rope_bwd")
    return r


def fa_kvcache_append_q8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens, *, q=None, q_out=None,
                         cu_seqlens_q=None, block_table=None, positions=None, inv_freq=None, mscale=1.0,
                         interleaved=False, q_weight=None, k_weight=None, eps=None, seqlens_out=None, workspace=None,
                         stream=None, event_begin=None, event_end=None):
    """fa_kvcache_append into a cache in 8 bits (fa_kvcache_append_q8 of the C
    ABI): ``k_cache`` and ``v_cache`` are torch.float8_e4m3fn, ``k_scale`` and
    ``v_scale`` fp32 [num_pages, page_size / block, Hkv].  With ``eps`` the rows
    of q and k are normalised first, with ``q_weight`` and ``k_weight``.  Returns
    ``(q_out, seqlens_out, workspace)`` as fa_kvcache_append; raises FaError on a
    non-zero status."""
    r = _binding.kvcache_append_q8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens, q, q_out, cu_seqlens_q,
                                   block_table, positions, inv_freq, mscale, interleaved, q_weight, k_weight, eps, seqlens_out,
                                   workspace, stream, _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_kvcache_append_q8")
    return r


def fa_kvcache_read_q8(k_cache, v_cache, k_scale, v_scale, seqlens_k=None, *, cu_seqlens_k=None, block_table=None,
                       total_k=None, max_seqlen_k=None, dtype=torch.bfloat16, k_out=None, v_out=None, workspace=None,
                       stream=None, event_begin=None, event_end=None):
    """Keys and values read back from a cache in 8 bits (fa_kvcache_read_q8 of
    the C ABI): packed [total_k, Hkv, d] with ``cu_seqlens_k`` and ``total_k``, or
    [n_seq, max_seqlen_k, Hkv, d] with ``seqlens_k`` and ``max_seqlen_k`` (rows
    past a sequence's keys are not written).  Returns ``(k_out, v_out,
    workspace)``, allocated with torch in ``dtype`` when not given; raises FaError
    on a non-zero status."""
    if dtype not in (torch.bfloat16, torch.float16):
        _raise(FA_ERR_INVALID_ARG, "fa_kvcache_read_q8 (dtype)")
    r = _binding.kvcache_read_q8(k_cache, v_cache, k_scale, v_scale, cu_seqlens_k, seqlens_k, block_table, k_out, v_out,
                                 max_seqlen_k if cu_seqlens_k is None else total_k, dtype == torch.float16, workspace, stream,
                                 _event(event_begin), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_kvcache_read_q8")
    return r


def fa_fwd_chunk_q8_plan(q, k_cache, v_cache, k_scale, v_scale, seqlens_k, *, out=None, lse=None, cu_seqlens_q=None,
                         block_table=None, prefix_lens=None, sink_keys=0, window_left=-1, window_right=-1, softcap=0.0,
                         scale=None, causal=True, max_seqlen_q=None, max_seqlen_k=None, debug_flags=0, **_):
    """Host-only plan query of fa_fwd_chunk_q8; returns (status, plan dict)."""
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]) if cu_seqlens_q is not None else (q.shape[0], q.shape[2], q.shape[1]),
                          dtype=torch.float32, device=q.device)
    plan = _lib.fa_plan()
    rc = _binding.fwd_chunk_q8_plan(q, k_cache, v_cache, k_scale, v_scale, q if out is None else out, lse, cu_seqlens_q, seqlens_k,
                                    block_table, prefix_lens, sink_keys, window_left, window_right, softcap, scale, causal,
                                    max_seqlen_q, max_seqlen_k, debug_flags, ctypes.addressof(plan))
    return rc, plan.as_dict()


def fa_fwd_chunk_q8(q, k_cache, v_cache, k_scale, v_scale, seqlens_k, *, out=None, lse=None, cu_seqlens_q=None,
                    block_table=None, prefix_lens=None, sink_keys=0, window_left=-1, window_right=-1, softcap=0.0, scale=None,
                    causal=True, max_seqlen_q=None, max_seqlen_k=None, workspace=None, stream=None, debug_flags=0,
                    event_begin=None, event_end=None, event_attn_end=None, alibi_slopes=None):
    """fa_fwd_chunk over a cache in 8 bits (fa_fwd_chunk_q8 of the C ABI), with
    the first ``sink_keys`` keys of a sequence exempt from ``window_left``.
    Arguments and results are otherwise those of fa_fwd_chunk."""
    r = _binding.fwd_chunk_q8(q, k_cache, v_cache, k_scale, v_scale, out, lse, cu_seqlens_q, seqlens_k, block_table, prefix_lens,
                              sink_keys, window_left, window_right, softcap, scale, causal, max_seqlen_q, max_seqlen_k, debug_flags,
                              stream, workspace, alibi_slopes, _event(event_begin), _event(event_attn_end), _event(event_end))
    if type(r) is int:
        _raise(r, "fa_fwd_chunk_q8")
    return r
