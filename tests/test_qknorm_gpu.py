"""GPU tests of fa_qk_norm_rope and fa_qk_norm_rope_bwd against the fp64 oracle."""
import numpy as np
import pytest
import torch

from norm_util import assert_grad, assert_normed
from oracle import qknorm as N

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, H = torch.bfloat16, torch.float16


def fa():
    import masked_flash_attention_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=BF, size=1.0):
    return (size * torch.randn(*shape, generator=g, dtype=torch.float32)).to(dtype)


def freqs(rot):
    return fa().fa_rope_inv_freq(rot)[0] if rot else None


def dev(t):
    return None if t is None else t.to(DEV)


def both(q, k, gq, gk, qw, kw, f, pos=None, **kwargs):
    """Forward and backward on the GPU and against the oracle."""
    m = fa()
    p = pos if pos is not None else None
    at = np.broadcast_to(np.arange(q.shape[1]), q.shape[:2]) if pos is None else pos.numpy()
    call = dict(q_weight=dev(qw), k_weight=dev(kw), inv_freq=dev(f), positions=dev(p), **kwargs)
    qo, ko = m.fa_qk_norm_rope(dev(q), dev(k), **call)
    dq, dk, dqw, dkw, ws = m.fa_qk_norm_rope_bwd(dev(gq), dev(gk), dev(q), dev(k), **call)
    for x, g, w, y, dx, dw in ((q, gq, qw, qo, dq, dqw), (k, gk, kw, ko, dk, dkw)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        assert (dw is None) == (w is None)
        assert_normed(y, x, at, f, w=w, **kwargs)
        assert_grad(dx, dw, g, x, at, f, w=w, **kwargs)
    return qo, ko, dq, dk, dqw, dkw


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 24), (64, 2), (64, 0), (128, 128), (128, 48), (128, 42), (128, 126), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,B,S,hq,hkv", [(BF, 2, 37, 6, 2), (H, 3, 1, 12, 12), (BF, 1, 130, 1, 1), (H, 1, 7, 40, 8)])
def test_values(d, rot, interleaved, dtype, B, S, hq, hkv):
    g = gen(rot + S)
    q, k, gq, gk = (rnd(g, B, S, h, d, dtype=dtype, size=3.0) for h in (hq, hkv, hq, hkv))
    qw, kw = 1 + 0.3 * torch.randn(d, generator=g), (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    both(q, k, gq, gk, qw, kw, freqs(rot), mscale=1.25 if rot else 1.0, interleaved=interleaved)


@pytest.mark.parametrize("rows", [1, 2, 151, 305, 911, 1217, 5001])  # each number of tokens per CTA, and a last part
@pytest.mark.parametrize("d", [64, 128])
def test_packed_rows_and_positions(rows, d):
    g = gen(rows)
    q, k, gq, gk = (rnd(g, rows, h, d) for h in (5, 2, 5, 2))
    pos = torch.randint(-100000, 1000000, (rows,), generator=g, dtype=torch.int32)
    f = torch.cat([freqs(d)[:4], torch.zeros(4, dtype=torch.float64)])  # (fp64 angles of the oracle stay exact enough)
    both(q, k, gq, gk, rnd(g, d), torch.ones(d), f, pos)


def test_without_k_weights_or_positions():
    g = gen(1)
    q, gq = rnd(g, 2, 9, 3, 64, dtype=H), rnd(g, 2, 9, 3, 64, dtype=H)
    both(q, None, gq, None, None, None, freqs(64))
    both(q, None, gq, None, None, None, None)
    both(q, q[:, :, :1].contiguous(), gq, gq[:, :, :1].contiguous(), None, torch.ones(64), None, eps=0.25)
    m = fa()
    # a weight's gradient without the weight (it stands for ones)
    dw = torch.full((64,), float("nan"), device=DEV)
    dq, _, dqw, _, ws = m.fa_qk_norm_rope_bwd(dev(gq), None, dev(q), dq_weight=dw)
    assert dqw is dw and ws is not None
    assert_grad(dq, dw, gq, q, None, None)
    assert m.fa_qk_norm_rope_bwd(dev(gq), None, dev(q))[2:] == (None, None, None)


@pytest.mark.parametrize("dtype", [BF, H])
def test_sizes_of_rows(dtype):
    """Rows of zeros, tiny and large rows, one large element."""
    g = gen(2)
    q = rnd(g, 1, 40, 2, 128, dtype=torch.float32)
    q[0, 0] = 0
    q[0, 1] *= 1e-4
    q[0, 2] *= 400
    q[0, 3, :, 77] = 30000.0
    q[0, 4] = 1.0
    q = q.to(dtype)
    gq = rnd(g, 1, 40, 2, 128, dtype=dtype)
    # (dx grows as 1 / |x|: without eps in the sum it would leave fp16)
    both(q, None, gq, None, rnd(g, 128, dtype=dtype), None, freqs(128), eps=1e-5)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (42, False)])
def test_in_place_and_strided(rot, interleaved):
    """q and k as slices of one fused projection, worked on where they are; v untouched."""
    g = gen(rot)
    fused, grads = rnd(g, 2, 70, 8, 128), rnd(g, 2, 70, 8, 128)
    qw, kw, f = rnd(g, 128), rnd(g, 128), freqs(rot)
    at = np.broadcast_to(np.arange(70), (2, 70))
    m = fa()
    kwargs = dict(q_weight=dev(qw), k_weight=dev(kw), inv_freq=dev(f), interleaved=interleaved)
    x, y = dev(fused), dev(grads)
    dq, dk, dqw, dkw, _ = m.fa_qk_norm_rope_bwd(y[:, :, :4], y[:, :, 4:6], x[:, :, :4], x[:, :, 4:6], dq=y[:, :, :4],
                                                dk=y[:, :, 4:6], **kwargs)
    for lo, hi, w, dw in ((0, 4, qw, dqw), (4, 6, kw, dkw)):
        assert_grad(y[:, :, lo:hi], dw, grads[:, :, lo:hi], fused[:, :, lo:hi], at, f, w=w, interleaved=interleaved)
    assert torch.equal(y[:, :, 6:].cpu(), grads[:, :, 6:]) and torch.equal(x.cpu(), fused)
    out = m.fa_qk_norm_rope(x[:, :, :4], x[:, :, 4:6], q_out=x[:, :, :4], k_out=x[:, :, 4:6], **kwargs)
    for lo, hi, w in ((0, 4, qw), (4, 6, kw)):
        assert_normed(x[:, :, lo:hi], fused[:, :, lo:hi], at, f, w=w, interleaved=interleaved)
    assert torch.equal(x[:, :, 6:].cpu(), fused[:, :, 6:]) and out[0].data_ptr() == x.data_ptr()
    # dq written over q, and [B, H, S, d] seen as [B, S, H, d]
    t, gt = rnd(g, 2, 3, 70, 128), rnd(g, 2, 3, 70, 128)
    z = dev(t).transpose(1, 2)
    dq = m.fa_qk_norm_rope_bwd(dev(gt).transpose(1, 2), None, z, dq=z, inv_freq=dev(f), interleaved=interleaved)[0]
    assert_grad(z, None, gt.transpose(1, 2), t.transpose(1, 2), at, f, interleaved=interleaved)


def test_nothing_to_do():
    m = fa()
    q = torch.empty(0, 3, 4, 64, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    assert m.fa_qk_norm_rope(q, q_weight=w)[0].shape == q.shape
    dq, _, dw, _, _ = m.fa_qk_norm_rope_bwd(q, None, q, q_weight=w, dq_weight=torch.full((64,), 3.0, device=DEV))
    assert dq.shape == q.shape and (dw == 0).all()


def test_nan_and_infinity_stay_in_their_rows():
    g = gen(4)
    q = rnd(g, 1, 20, 4, 64)
    q[0, 3, 1, 5], q[0, 7, 2, 60] = float("nan"), float("inf")
    y, _ = fa().fa_qk_norm_rope(dev(q), inv_freq=dev(freqs(64)))
    bad = torch.zeros(1, 20, 4, dtype=torch.bool)
    bad[0, 3, 1] = bad[0, 7, 2] = True
    assert torch.isfinite(y.cpu()[~bad]).all()
    assert torch.isnan(y.cpu()[0, 3, 1]).all()
    clean = q.clone()
    clean[0, 3, 1], clean[0, 7, 2] = 0, 0
    y2, _ = fa().fa_qk_norm_rope(dev(clean), inv_freq=dev(freqs(64)))
    assert torch.equal(y.cpu()[~bad], y2.cpu()[~bad])


def test_same_bits_again():
    g = gen(5)
    q, k, gq, gk = (rnd(g, 3, 500, h, 128) for h in (8, 2, 8, 2))
    w = rnd(g, 128)
    a = both(q, k, gq, gk, w, w, freqs(128))
    b = both(q, k, gq, gk, w, w, freqs(128))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_norm_then_rotation_is_the_two_operators():
    """Against fa_rope of the normalised rows, which are rounded on the way there."""
    g = gen(6)
    q = rnd(g, 1, 300, 4, 128, dtype=H)
    f = dev(freqs(128))
    y, _ = fa().fa_qk_norm_rope(dev(q), inv_freq=f, mscale=1.1)
    n, _ = fa().fa_qk_norm_rope(dev(q))
    z, _ = fa().fa_rope(n, inv_freq=f, mscale=1.1)
    ref = np.abs(N.norm(q)).max()
    # two roundings of the pair and two of the results, each half a step of fp16
    assert (y.double() - z.double()).abs().max().item() <= 1.1 * ref * (2 * 2.0 ** -11 + 2 * 2 ** 0.5 * 2.0 ** -11)


def test_gradient_through_the_attention():
    """Projections -> norm and rotation -> fa_fwd -> loss, and back: fa_bwd's dq and dk through
    fa_qk_norm_rope_bwd, against differences of the fp64 loss."""
    from oracle import attention as A
    m = fa()
    g = gen(7)
    B, S, hq, hkv, d = 1, 140, 4, 2, 64
    q, k, v, dout = (rnd(g, B, S, h, d) for h in (hq, hkv, hkv, hq))
    qw, kw, f = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g), freqs(d)
    kwargs = dict(q_weight=dev(qw), k_weight=dev(kw), inv_freq=dev(f))
    qn, kn = m.fa_qk_norm_rope(dev(q), dev(k), **kwargs)
    out, lse, _ = m.fa_fwd(qn, kn, dev(v), causal=True)
    gq, gk, _, _ = m.fa_bwd(qn, kn, dev(v), out, lse, dev(dout), causal=True)
    dq, dk, dqw, dkw, _ = m.fa_qk_norm_rope_bwd(gq, gk, dev(q), dev(k), **kwargs)
    pos = np.arange(S)[None]

    def loss(q, k, qw, kw):
        o, _ = A.attention(N.norm_rope(q, pos, f, w=qw), N.norm_rope(k, pos, f, w=kw), v, causal=True)
        return (o * dout.double().numpy()).sum()

    x = [q.double().numpy(), k.double().numpy(), qw.double().numpy(), kw.double().numpy()]
    got = [t.double().cpu().numpy() for t in (dq, dk, dqw, dkw)]
    for n, ats in ((0, [(0, 100, 1, 3), (0, 139, 3, 20)]), (1, [(0, 60, 1, 17), (0, 5, 0, 40)]), (2, [(7,), (40,)]), (3, [(0,), (63,)])):
        for at in ats:
            e = np.zeros_like(x[n])
            e[at] = 1e-4
            hi, lo = ([y + s * e if i == n else y for i, y in enumerate(x)] for s in (1, -1))
            ref = (loss(*hi) - loss(*lo)) / 2e-4
            # bf16 products through fa_bwd: the backward's own bound is 1e-2 of the whole gradient
            assert abs(got[n][at] - ref) <= 2e-2 * np.sqrt((got[n] ** 2).mean()) + 2e-2 * abs(ref), (n, at, got[n][at], ref)


def test_capture_and_other_stream():
    m = fa()
    g = gen(8)
    q, gq = dev(rnd(g, 1, 300, 4, 128)), dev(rnd(g, 1, 300, 4, 128))
    w, f = dev(rnd(g, 128)), dev(freqs(128))
    ws = torch.zeros(m._lib.FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)

    def step():
        y, _ = m.fa_qk_norm_rope(q, q_weight=w, inv_freq=f)
        return y, *m.fa_qk_norm_rope_bwd(gq, None, q, q_weight=w, inv_freq=f, workspace=ws)[::2][:2]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    q.copy_(rnd(g, 1, 300, 4, 128))
    graph.replay()
    torch.cuda.synchronize()
    now = step()
    assert all(torch.equal(a, b) for a, b in zip(got, now))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = m.fa_qk_norm_rope(q, q_weight=w, inv_freq=f, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, now[0])


def test_binding_refusals_on_the_device():
    m = fa()
    q = torch.zeros(1, 4, 2, 64, dtype=BF, device=DEV)
    for call in (lambda: m.fa_qk_norm_rope(q, q_weight=torch.ones(64)), lambda: m.fa_qk_norm_rope(q, k_weight=q[0, 0, 0]),
                 lambda: m.fa_qk_norm_rope(q, eps=0.0), lambda: m.fa_qk_norm_rope_bwd(q, q, q),
                 lambda: m.fa_qk_norm_rope_bwd(q, None, q, q_weight=q[0, 0, 0], workspace=q)):
        with pytest.raises(m.FaError):
            call()
    with pytest.raises(TypeError):
        m.fa_qk_norm_rope(q, eps=None)


@pytest.mark.parametrize("rows,hq,hkv,d", [(1000, 32, 8, 128), (700, 13, 3, 64), (9000, 9, 1, 64), (6500, 12, 3, 128)])
def test_shares_of_warps(rows, hq, hkv, d):
    """Some rounds of a token to a warp, a whole token, and a last round that is not full; several rounds to a warp of the gradient."""
    g = gen(rows)
    q, k, gq, gk = (rnd(g, rows, h, d) for h in (hq, hkv, hq, hkv))
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32)
    both(q, k, gq, gk, rnd(g, d), rnd(g, d), freqs(d), pos)


@pytest.mark.parametrize("half", [False, True])
def test_weights_at_any_address(half):
    """Weights that begin off a 16-byte boundary."""
    g = gen(9)
    q, gq = rnd(g, 1, 33, 5, 128), rnd(g, 1, 33, 5, 128)
    base = rnd(g, 132) if half else torch.randn(132, generator=g)
    m = fa()
    for off in (1, 3):
        w = dev(base)[off:off + 128]
        y, _ = m.fa_qk_norm_rope(dev(q), q_weight=w, inv_freq=dev(freqs(128)))
        dq, _, dw, _, _ = m.fa_qk_norm_rope_bwd(dev(gq), None, dev(q), q_weight=w, inv_freq=dev(freqs(128)))
        at = np.arange(33)[None]
        assert_normed(y, q, at, freqs(128), w=base[off:off + 128])
        assert_grad(dq, dw, gq, q, at, freqs(128), w=base[off:off + 128])


def test_broadcast_gradient():
    """One dy row for all heads and tokens (strides of 0)."""
    g = gen(10)
    q, gq = rnd(g, 2, 30, 6, 64, dtype=H), rnd(g, 1, 1, 1, 64, dtype=H)
    dq, _, dw, _, _ = fa().fa_qk_norm_rope_bwd(dev(gq).expand(2, 30, 6, 64), None, dev(q), q_weight=dev(torch.ones(64)), inv_freq=dev(freqs(64)))
    assert_grad(dq, dw, gq.expand(2, 30, 6, 64).contiguous(), q, np.broadcast_to(np.arange(30), (2, 30)), freqs(64), w=torch.ones(64))


def test_infinite_gradient_reaches_its_column():
    """An infinite dy makes its column of dw infinite or NaN, no other."""
    g = gen(11)
    q, gq = rnd(g, 1, 50, 4, 64), rnd(g, 1, 50, 4, 64)
    gq[0, 20, 1, 7] = float("inf")
    dq, _, dw, _, _ = fa().fa_qk_norm_rope_bwd(dev(gq), None, dev(q), q_weight=dev(torch.ones(64)))
    bad = ~torch.isfinite(dw.cpu())
    assert bad[7] and bad.sum() == 1
    rows = ~torch.isfinite(dq.cpu()).all(-1)
    assert rows[0, 20, 1] and rows.sum() == 1


def test_two_streams_at_once():
    """Gradients of two layers on two streams, each with its own workspace."""
    m = fa()
    g = gen(12)
    layers = [tuple(dev(rnd(g, 1, 2000, h, 128)) for h in (8, 2, 8, 2)) for _ in range(2)]
    w, f = dev(rnd(g, 128)), dev(freqs(128))
    one = [m.fa_qk_norm_rope_bwd(a, b, c, d, q_weight=w, k_weight=w, inv_freq=f)[:4] for a, b, c, d in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(5):
        for i, (s, (a, b, c, d)) in enumerate(zip(streams, layers)):
            with torch.cuda.stream(s):
                got[i] = m.fa_qk_norm_rope_bwd(a, b, c, d, q_weight=w, k_weight=w, inv_freq=f)[:4]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a, b in zip(one, got) for x, y in zip(a, b))
