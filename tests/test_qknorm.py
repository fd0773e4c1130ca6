"""Norms of queries and keys on the CPU: pins of the oracle and the refusals of
fa_qk_norm_rope and fa_qk_norm_rope_bwd (found on the host before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import masked_flash_attention_gb300 as fa
from masked_flash_attention_gb300 import _lib
from oracle import qknorm as N
from oracle import rotary as R

BF, H = torch.bfloat16, torch.float16
E = _lib.FA_ERR_INVALID_ARG


def _rows(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_oracle_rows_have_unit_mean_square():
    x = 7.0 * _rows(0, 5, 3, 64)
    y = N.norm(x, eps=1e-12)
    assert np.allclose((y * y).mean(-1), 1.0) and np.allclose(y * x, np.abs(y * x))
    w = _rows(1, 64)
    assert np.allclose(N.norm(x, w, 1e-12), y * w)
    # eps alone decides a row of zeros, and bounds tiny ones
    assert (N.norm(np.zeros((1, 64))) == 0).all()
    assert np.allclose(N.norm(np.full((1, 64), 1e-3), eps=1e-6), 1e-3 / np.sqrt(2e-6))
    f = 100.0 ** (-np.arange(16) / 16)
    assert np.array_equal(N.norm_rope(x, np.arange(5), f, w=w), R.rope(N.norm(x, w), np.arange(5), f))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [1e-6, 0.5])
def test_oracle_gradient_by_differences(interleaved, eps):
    f = 50.0 ** (-np.arange(12) / 12)
    x, g, w = _rows(2, 4, 2, 64), _rows(3, 4, 2, 64), 1 + 0.3 * _rows(4, 64)
    pos, kw = np.array([0, 3, 50, -2]), dict(eps=eps, mscale=1.25, interleaved=interleaved)
    loss = lambda x, w: (g * N.norm_rope(x, pos, f, w=w, **kw)).sum()  # noqa: E731
    dx, dw = N.norm_rope_grad(g, x, pos, f, w=w, **kw)
    h = 1e-5
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 13), (3, 1, 23), (1, 0, 40)]:
        e = np.zeros_like(x)
        e[at] = h
        assert np.isclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[at], rtol=1e-7, atol=1e-8)
        e = np.zeros(64)
        e[at[-1]] = h
        assert np.isclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[at[-1]], rtol=1e-7, atol=1e-8)


def T(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _call(fn, tensors, scalars, opts=None):
    descs = [_lib.describe(t) for t in tensors]
    opts = _lib.make_opts(stream=0) if opts is None else opts
    return fn(*[ctypes.byref(x) if x is not None else None for x in descs], *scalars, ctypes.byref(opts))


def like(t):
    return None if t is None else T(*t.shape, dtype=t.dtype)


def fwd_rc(q, k=None, qw=None, kw=None, q_out="like", k_out="like", positions=None, inv_freq=None, eps=1e-6, mscale=1.0):
    q_out = like(q) if isinstance(q_out, str) else q_out
    k_out = like(k) if isinstance(k_out, str) else k_out
    return _call(fa.lib.fa_qk_norm_rope, (q, k, qw, kw, q_out, k_out, positions, inv_freq), [eps, mscale, 0])


def bwd_rc(q, k=None, gq="like", gk="like", qw=None, kw=None, dq="like", dk="like", dqw=None, dkw=None, positions=None,
           inv_freq=None, eps=1e-6, mscale=1.0, ws=0):
    gq, gk, dq, dk = (like(x) if isinstance(y, str) else y for x, y in ((q, gq), (k, gk), (q, dq), (k, dk)))
    opts = _lib.make_opts(stream=0)
    if ws:
        opts.workspace, opts.workspace_bytes = 256, ws
    return _call(fa.lib.fa_qk_norm_rope_bwd, (gq, gk, q, k, qw, kw, dq, dk, dqw, dkw, positions, inv_freq), [eps, mscale, 0], opts)


def shared_refusals(rc):
    q, k = T(2, 5, 4, 64), T(2, 5, 2, 64)
    i32 = lambda *s: T(*s, dtype=torch.int32)  # noqa: E731
    f64 = lambda *s: T(*s, dtype=torch.float64)  # noqa: E731
    return [
        rc(q.float()), rc(T(2, 5, 4, 96)), rc(T(2, 5, 4, 256)), rc(T(5, 64)), rc(q, k.half()), rc(q, T(2, 6, 2, 64)),
        rc(q, T(2, 5, 0, 64)), rc(q, T(10, 2, 64)), rc(T(2, 5, 4, 68)[..., :64]), rc(T(2, 5, 4, 128)[..., ::2]),
        rc(q, qw=T(63)), rc(q, qw=T(64).half()), rc(q, qw=f64(64)), rc(q, qw=T(1, 64)), rc(q, qw=T(128)[::2]), rc(q, kw=T(64)),
        rc(q, k, kw=T(32)),
        rc(q, inv_freq=f64(33)), rc(q, inv_freq=f64(0)), rc(q, inv_freq=T(16, dtype=torch.float32)), rc(q, inv_freq=f64(32)[::2]),
        rc(q, inv_freq=f64(16), mscale=float("nan")), rc(q, inv_freq=f64(16), mscale=float("inf")),
        rc(T(10, 4, 64), inv_freq=f64(16)), rc(T(10, 4, 64), inv_freq=f64(16), positions=i32(2, 5)),
        rc(q, inv_freq=f64(16), positions=i32(2, 4)), rc(q, inv_freq=f64(16), positions=i32(2, 5).long()),
        rc(q, eps=0.0), rc(q, eps=-1e-6), rc(q, eps=float("nan")), rc(q, eps=float("inf")),
    ]


def test_forward_refusals():
    q, k = T(2, 5, 4, 64), T(2, 5, 2, 64)
    bad = shared_refusals(fwd_rc) + [
        fwd_rc(q, q_out=None), fwd_rc(q, q_out=T(2, 5, 2, 64)), fwd_rc(q, q_out=q.half()), fwd_rc(q, k, k_out=None),
        fwd_rc(q, k_out=k), fwd_rc(q, q_out=T(1, 5, 4, 64).expand(2, 5, 4, 64)),
    ]
    assert bad == [E] * len(bad), bad


def test_backward_refusals():
    q, k = T(2, 5, 4, 64), T(2, 5, 2, 64)
    f32 = lambda *s: T(*s, dtype=torch.float32)  # noqa: E731
    bad = shared_refusals(bwd_rc) + [
        bwd_rc(q, gq=None), bwd_rc(q, gq=q.half()), bwd_rc(q, gq=T(2, 5, 2, 64)), bwd_rc(q, gk=k), bwd_rc(q, k, gk=None),
        bwd_rc(q, k, dk=None), bwd_rc(q, dq=None), bwd_rc(q, dq=T(2, 5, 2, 64)), bwd_rc(q, dq=T(1, 5, 4, 64).expand(2, 5, 4, 64)),
        bwd_rc(q, dqw=T(64)), bwd_rc(q, dqw=f32(32)), bwd_rc(q, dqw=f32(128)[::2]), bwd_rc(q, dkw=f32(64)),
    ]
    assert bad == [E] * len(bad), bad
    need = _lib.FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES
    assert bwd_rc(q, k, dqw=f32(64)) == bwd_rc(q, k, dkw=f32(64), ws=need - 1) == _lib.FA_ERR_WORKSPACE


def test_bindings_refuse_host_tensors_and_odd_arguments():
    q = T(1, 2, 2, 64)
    for call in (lambda: fa.fa_qk_norm_rope(q), lambda: fa.fa_qk_norm_rope_bwd(q, None, q)):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.status == E
    with pytest.raises(fa.FaError):
        fa.fa_qk_norm_rope(None)


def test_workspace_size_of_the_header():
    import os
    import re
    txt = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa.h")).read()
    m = re.search(r"#define FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES \(\(size_t\)256 \+ \(\(size_t\)1 << (\d+)\)\)", txt)
    assert 256 + (1 << int(m.group(1))) == _lib.FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES
