"""Rotary positions on the CPU: pins of the oracle, the frequencies of scaled
embeddings, and the refusals of fa_rope and fa_kvcache_append (argument errors
are found on the host before any device work)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import masked_flash_attention_gb300 as fa
from masked_flash_attention_gb300 import _lib
from oracle import rotary as R

BF = torch.bfloat16
E = _lib.FA_ERR_INVALID_ARG


def _rows(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [2, 24, 64])
def test_oracle_pairs_turn_by_their_angle(interleaved, rot):
    f = 1000.0 ** (-np.arange(rot // 2) / (rot // 2))
    x = _rows(0, 3, 2, 64)
    y = R.rope(x, [0, 7, -3], f, mscale=1.5, interleaved=interleaved)
    assert np.array_equal(y[0][:, rot:], x[0][:, rot:]) and np.allclose(y[0][:, :rot], 1.5 * x[0][:, :rot])
    for r, p in ((1, 7), (2, -3)):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = math.cos(p * f[i]), math.sin(p * f[i])
            assert np.allclose(y[r][:, a], 1.5 * (x[r][:, a] * c - x[r][:, b] * s))
            assert np.allclose(y[r][:, b], 1.5 * (x[r][:, a] * s + x[r][:, b] * c))


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_scores_depend_on_the_distance_alone(interleaved):
    f = 10000.0 ** (-np.arange(32) / 32)
    q, k = _rows(1, 1, 64), _rows(2, 1, 64)
    at = lambda x, p: R.rope(x, p, f, interleaved=interleaved)  # noqa: E731
    ref = (at(q, 5) * at(k, 2)).sum()
    assert np.isclose((at(q, 1005) * at(k, 1002)).sum(), ref)
    assert not np.isclose((at(q, 1005) * at(k, 1003)).sum(), ref)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_inverse_is_the_gradient(interleaved):
    """d <g, rope(x)> / dx = inverse rope of g, by central differences (the map
    is linear, so they are exact but for rounding)."""
    f = 100.0 ** (-np.arange(12) / 12)
    x, g = _rows(3, 4, 2, 64), _rows(4, 4, 2, 64)
    pos = np.array([0, 3, 50, -2])
    kw = dict(mscale=1.25, interleaved=interleaved)
    grad = R.rope(g, pos, f, inverse=True, **kw)
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 13), (3, 1, 23), (1, 0, 40)]:
        e = np.zeros_like(x)
        e[at] = 0.5
        num = (g * (R.rope(x + e, pos, f, **kw) - R.rope(x - e, pos, f, **kw))).sum()
        assert np.isclose(num, grad[at], rtol=1e-10, atol=1e-12)


def test_oracle_append_without_rotation_is_the_plain_append():
    from oracle import kvcache as K
    rng = np.random.default_rng(5)
    kn, vn = rng.standard_normal((5, 2, 64)), rng.standard_normal((5, 2, 64))
    kc, vc = rng.standard_normal((6, 4, 2, 64)), rng.standard_normal((6, 4, 2, 64))
    bt = np.array([[3, 1], [0, 5]])
    a = R.kvcache_append(kn, vn, kc, vc, [3, 2], cu_seqlens_q=[0, 2, 5], block_table=bt)
    b = K.append_kvcache(kc, vc, kn, vn, [3, 2], cu_seqlens_q=[0, 2, 5], block_table=bt)
    assert np.array_equal(a[1], b[0]) and np.array_equal(a[2], b[1]) and list(a[3]) == [5, 5]


# ---- frequencies ----

def test_plain_and_linear_frequencies():
    f, m = fa.fa_rope_inv_freq(64, 10000.0)
    ref = np.array([10000.0 ** (-2 * i / 64) for i in range(32)])
    assert m == 1.0 and np.allclose(f.numpy(), ref, rtol=1e-14)
    g, m = fa.fa_rope_inv_freq(64, 10000.0, scaling="linear", factor=4.0)
    assert m == 1.0 and np.allclose(g.numpy(), ref / 4, rtol=1e-14)


def test_ntk_keeps_the_highest_and_divides_the_lowest():
    f, _ = fa.fa_rope_inv_freq(128, 10000.0)
    g, _ = fa.fa_rope_inv_freq(128, 10000.0, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and np.isclose(float(f[-1] / g[-1]), 8.0, rtol=1e-12)


def test_blend_frequencies():
    kw = dict(scaling="blend", factor=8.0, original_len=8192, low=1.0, high=4.0)
    f, _ = fa.fa_rope_inv_freq(128, 500000.0)
    g, m = fa.fa_rope_inv_freq(128, 500000.0, **kw)
    assert m == 1.0
    turns = 8192 * f.numpy() / (2 * math.pi)
    fast, slow = turns >= 4.0, turns <= 1.0
    assert fast.any() and slow.any() and not (fast | slow).all()
    assert np.array_equal(g.numpy()[fast], f.numpy()[fast]) and np.allclose(g.numpy()[slow], f.numpy()[slow] / 8, rtol=1e-14)
    w = (turns - 1) / 3
    mid = ~(fast | slow)
    assert np.allclose(g.numpy()[mid], (w * f.numpy() + (1 - w) * f.numpy() / 8)[mid], rtol=1e-13)


def test_yarn_frequencies():
    f, _ = fa.fa_rope_inv_freq(128, 10000.0)
    g, m = fa.fa_rope_inv_freq(128, 10000.0, scaling="yarn", factor=16.0, original_len=4096, low=1.0, high=32.0)
    assert np.isclose(m, 0.1 * math.log(16.0) + 1.0)
    idx = lambda n: 128 * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = math.floor(idx(32.0)), math.ceil(idx(1.0))
    share = 1 - np.clip((np.arange(64) - lo) / (hi - lo), 0, 1)
    assert np.allclose(g.numpy(), share * f.numpy() + (1 - share) * f.numpy() / 16, rtol=1e-13)
    # the bounds in turns: pairs that turn 32 times or more are kept, once or less divided
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert np.array_equal(g.numpy()[turns >= 33], f.numpy()[turns >= 33])


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(rot=64, base=1.0), dict(rot=64, base=float("nan")),
                                dict(rot=64, scaling="linear", factor=0.5), dict(rot=64, scaling="linear", factor=float("inf")),
                                dict(rot=2, scaling="ntk", factor=2.0), dict(rot=64, scaling="blend", factor=2.0),
                                dict(rot=64, scaling="blend", factor=2.0, original_len=100, low=4.0, high=1.0),
                                dict(rot=64, scaling="yarn", factor=2.0, original_len=100, low=0.0, high=1.0),
                                dict(rot=64, scaling="other")])
def test_frequency_refusals(kw):
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope_inv_freq(**kw)
    assert e.value.status == E


# ---- refusals: raw calls of the C entry points with host tensors; every one
# is refused before the device is looked at ----

def T(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _call(fn, tensors, mid, opts, last=None):
    descs = [_lib.describe(t) for t in tensors]
    args = [ctypes.byref(x) if x is not None else None for x in descs] + mid
    if last is not None:
        tail = _lib.describe(last[0])
        args.append(ctypes.byref(tail) if tail is not None else None)
    return fn(*args, ctypes.byref(opts) if opts is not None else None)


def rope_rc(q, k=None, q_out="like", k_out="like", positions=None, inv_freq=None, mscale=1.0):
    q_out = T(*q.shape, dtype=q.dtype) if isinstance(q_out, str) else q_out
    k_out = (None if k is None else T(*k.shape, dtype=k.dtype)) if isinstance(k_out, str) else k_out
    inv_freq = T(16, dtype=torch.float64) if inv_freq is None else inv_freq
    return _call(fa.lib.fa_rope, (q, k, q_out, k_out, positions, inv_freq), [mscale, 0, 0], _lib.make_opts(stream=0))


def test_rope_refusals():
    q, k = T(2, 5, 4, 64), T(2, 5, 2, 64)
    i32 = lambda *s: T(*s, dtype=torch.int32)  # noqa: E731
    bad = [
        rope_rc(q.float()), rope_rc(T(2, 5, 4, 96)), rope_rc(T(2, 5, 4, 256)), rope_rc(T(5, 64)),
        rope_rc(q, k.half()), rope_rc(q, T(2, 6, 2, 64)), rope_rc(q, T(2, 5, 0, 64)), rope_rc(q, T(10, 2, 64)),
        rope_rc(q, q_out=T(2, 5, 2, 64)), rope_rc(q, q_out=q.half()), rope_rc(q, k, k_out=T(2, 5, 4, 64)),
        rope_rc(q, k, k_out=None), rope_rc(q, q_out=T(1, 5, 4, 64).expand(2, 5, 4, 64)),
        rope_rc(q, q_out=T(2, 5, 4, 128)[..., ::2]), rope_rc(q, q_out=T(2, 5, 4, 68)[..., :64]),
        rope_rc(q, inv_freq=T(33, dtype=torch.float64)), rope_rc(q, inv_freq=T(0, dtype=torch.float64)),
        rope_rc(q, inv_freq=T(16, dtype=torch.float32)), rope_rc(q, inv_freq=T(32, dtype=torch.float64)[::2]),
        rope_rc(q, inv_freq=T(4, 4, dtype=torch.float64)),
        rope_rc(q, positions=i32(2, 4)), rope_rc(q, positions=i32(5)), rope_rc(q, positions=T(2, 5, dtype=torch.int64)),
        rope_rc(T(10, 4, 64)), rope_rc(T(10, 4, 64), positions=i32(2, 5)),
        rope_rc(q, mscale=float("nan")), rope_rc(q, mscale=float("inf")),
    ]
    assert bad == [E] * len(bad), bad


def append_rc(kn=None, vn=None, kc=None, vc=None, lens=None, q=None, q_out=None, cu=None, bt=None, positions=None,
              inv_freq=None, mscale=1.0, out=None, ws=True):
    kn = T(2, 3, 2, 64) if kn is None else kn
    vn = kn if vn is None else vn
    kc = T(2, 9, 2, 64) if kc is None else kc
    vc = T(*kc.shape, dtype=kc.dtype) if vc is None else vc
    lens = T(2, dtype=torch.int32) if lens is None else lens
    opts = _lib.make_opts(stream=0)
    if ws:
        opts.workspace, opts.workspace_bytes = 256, 256
    return _call(fa.lib.fa_kvcache_append, (q, q_out, kn, vn, kc, vc, cu, lens, bt, positions, inv_freq), [mscale, 0],
                 opts, (out,))


def test_append_refusals():
    i32 = lambda *s: T(*s, dtype=torch.int32)  # noqa: E731
    pages, bt = T(8, 4, 2, 64), i32(2, 3)
    q = T(2, 3, 4, 64)
    lens2 = i32(4)
    bad = [
        append_rc(kn=T(2, 3, 2, 96)), append_rc(kn=T(2, 3, 2, 64).float()), append_rc(kn=T(6, 2, 64)),
        append_rc(vn=T(2, 3, 1, 64)), append_rc(vn=T(2, 3, 2, 64).half()),
        append_rc(kc=T(3, 9, 2, 64)), append_rc(kc=T(2, 9, 4, 64)), append_rc(kc=T(2, 9, 2, 128)),
        append_rc(kc=T(2, 9, 2, 64).half()), append_rc(vc=T(2, 8, 2, 64)),
        append_rc(kc=T(2, 1, 2, 64).expand(2, 9, 2, 64)), append_rc(vc=T(1, 9, 2, 64).expand(2, 9, 2, 64)),
        append_rc(lens=i32(3)), append_rc(lens=T(2, dtype=torch.int64)),
        append_rc(kc=pages, bt=i32(3, 3)), append_rc(kc=pages, bt=i32(2, 0)), append_rc(kc=pages, bt=bt.long()),
        append_rc(kc=pages, bt=i32(3, 2).T), append_rc(kc=T(8, 0, 2, 64), bt=bt),
        append_rc(q=q), append_rc(q_out=q), append_rc(q=q, q_out=T(2, 3, 2, 64)), append_rc(q=q.half(), q_out=q.half()),
        append_rc(q=T(2, 4, 4, 64), q_out=T(2, 4, 4, 64)), append_rc(q=T(6, 4, 64), q_out=T(6, 4, 64)),
        append_rc(positions=i32(2, 2)), append_rc(positions=i32(6)),
        append_rc(inv_freq=T(33, dtype=torch.float64)), append_rc(inv_freq=T(8, dtype=torch.float64), mscale=float("nan")),
        append_rc(out=i32(3)), append_rc(lens=lens2[:2], out=lens2[1:3]), append_rc(lens=lens2[:2], out=lens2[:2]),
        append_rc(kn=T(6, 2, 64), cu=i32(3, 1)), append_rc(kn=T(6, 2, 64), cu=i32(4)),
        append_rc(kn=T(2, 3, 2, 64), cu=i32(3)),
    ]
    assert bad == [E] * len(bad), bad
    assert append_rc(ws=False) == _lib.FA_ERR_WORKSPACE


def test_bindings_refuse_host_tensors():
    q, f = T(1, 2, 2, 64), T(8, dtype=torch.float64)
    with pytest.raises(fa.FaError):
        fa.fa_rope(q, inv_freq=f)
    with pytest.raises(fa.FaError):
        fa.fa_kvcache_append(q, q, q, q, T(1, dtype=torch.int32))


@pytest.mark.parametrize("kw", [dict(rot=64, scaling="yarn", factor=2.0, original_len=2**32 + 8192, high=32.0),
                                dict(rot=64, scaling="blend", factor=2.0, original_len=2**31),
                                dict(rot=4, scaling="ntk", factor=1e200), dict(rot=2**32 + 64), dict(rot=-2**32 + 64)])
def test_frequency_arguments_past_their_range(kw):
    """Whole numbers past 32 bits wrapped, and a base past fp64 gave frequencies of zero."""
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope_inv_freq(**kw)
    assert e.value.status == E
