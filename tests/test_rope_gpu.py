"""GPU tests of fa_rope and fa_kvcache_append against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import rotary as R
from rope_util import assert_rotated

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, H = torch.bfloat16, torch.float16


def fa():
    import masked_flash_attention_gb300 as m
    return m


def rnd(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(dtype)


def freqs(rot, base=10000.0):
    return fa().fa_rope_inv_freq(rot, base)[0]


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 24), (64, 2), (128, 128), (128, 96), (128, 48), (128, 42),
                                   (128, 126)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,inverse,B,S,hq,hkv", [(BF, False, 2, 37, 6, 2), (H, True, 3, 1, 12, 12), (BF, True, 1, 130, 1, 1)])
def test_rope(d, rot, interleaved, dtype, inverse, B, S, hq, hkv):
    g = gen(rot + S)
    q, k = rnd(g, B, S, hq, d, dtype=dtype), rnd(g, B, S, hkv, d, dtype=dtype)
    f = freqs(rot)
    qo, ko = fa().fa_rope(q.to(DEV), k.to(DEV), inv_freq=f.to(DEV), mscale=1.25, interleaved=interleaved, inverse=inverse)
    pos = np.broadcast_to(np.arange(S), (B, S))
    for x, y in ((q, qo), (k, ko)):
        ref = R.rope(x, pos, f, mscale=1.25, interleaved=interleaved, inverse=inverse)
        assert_rotated(y, ref, x, f, 1.25, interleaved)


@pytest.mark.parametrize("rows", [1, 2, 151, 1217, 5000])  # each number of tokens per CTA and a last part
def test_rope_packed_far_and_negative_positions(rows):
    g = gen(rows)
    q, k = rnd(g, rows, 5, 128), rnd(g, rows, 2, 128)
    pos = torch.randint(-2**31, 2**31 - 1, (rows,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = 2**31 - 1
    f = freqs(128, 500000.0)
    qo, ko = fa().fa_rope(q.to(DEV), k.to(DEV), inv_freq=f.to(DEV), positions=pos.to(DEV))
    # the oracle's p * f in fp64 is itself off by 2^-53 * 2^31 rad, 2.4e-7, far out: the fp64 product is
    # reduced exactly here instead, from the frequency in units of 2^-200 turn
    import fractions
    import math
    two_pi = fractions.Fraction(6283185307179586476925286766559005768394338798750211641949889184615, 10**66)
    n = min(rows, 40)
    ang = np.array([[float((int(p) * fractions.Fraction(float(x)) / two_pi) % 1) * 2 * math.pi for x in f] for p in pos[:n]])
    z = np.exp(1j * ang)[:, None, :]
    for x, y in ((q[:n], qo[:n]), (k[:n], ko[:n])):
        xs = x.double().numpy()
        w = (xs[..., :64] + 1j * xs[..., 64:]) * z
        assert_rotated(y, np.concatenate([w.real, w.imag], -1), x, f, 1.0, False)
    # every later row: within the fp64 oracle's own doubt
    ref = R.rope(q, pos.numpy(), f)
    assert np.abs(qo.double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-5


def test_rope_frequencies_of_any_size():
    """Above a turn per position, negative, tiny and zero."""
    f = torch.tensor([1.0, 3.0, 100.0, -0.7, -5.0, 1e-7, 1e-300, 0.0, 2.0**40 + 0.25, 0.5, 2.0, 4.0], dtype=torch.float64)
    g = gen(3)
    q = rnd(g, 1, 300, 3, 64)
    for il in (False, True):
        qo, _ = fa().fa_rope(q.to(DEV), inv_freq=f.to(DEV), interleaved=il)
        ref = R.rope(q, np.arange(300)[None], f, interleaved=il)
        cols = [i for i in range(12) if abs(f[i]) < 2.0**20]  # at 2^40 rad per position fp64 has no angle left
        a, b = R.pairs(12, il)
        got = qo.cpu()
        keep = np.ones(64, bool)
        keep[[a[8], b[8]]] = False
        assert cols == [i for i in range(12) if i != 8]
        got2, ref2 = got.clone(), ref.copy()
        got2[..., ~torch.from_numpy(keep)] = 0
        ref2[..., ~keep] = 0
        assert_rotated(got2, ref2, q, f, 1.0, il)
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (42, False)])
def test_rope_in_place_and_strided(rot, interleaved):
    """q and k as slices of one fused projection, rotated where they are; v untouched."""
    g = gen(rot)
    fused = rnd(g, 2, 70, 4 + 2 + 2, 128)
    f = freqs(rot)
    dev = fused.to(DEV)
    q, k = dev[:, :, :4], dev[:, :, 4:6]
    pos = torch.randint(0, 5000, (1, 70), generator=g, dtype=torch.int32)
    out = fa().fa_rope(q, k, inv_freq=f.to(DEV), positions=pos.to(DEV).expand(2, 70), q_out=q, k_out=k, interleaved=interleaved)
    assert out[0] is q and out[1] is k
    p = pos.expand(2, 70).numpy()
    assert_rotated(dev[:, :, :4], R.rope(fused[:, :, :4], p, f, interleaved=interleaved), fused[:, :, :4], f, 1.0, interleaved)
    assert_rotated(dev[:, :, 4:6], R.rope(fused[:, :, 4:6], p, f, interleaved=interleaved), fused[:, :, 4:6], f, 1.0, interleaved)
    assert torch.equal(dev[:, :, 6:].cpu(), fused[:, :, 6:])
    # [B, H, S, d] seen as [B, S, H, d]
    t = rnd(g, 2, 3, 70, 128)
    y, _ = fa().fa_rope(t.to(DEV).transpose(1, 2), inv_freq=f.to(DEV), interleaved=interleaved)
    assert_rotated(y, R.rope(t.transpose(1, 2), np.broadcast_to(np.arange(70), (2, 70)), f, interleaved=interleaved),
                   t.transpose(1, 2), f, 1.0, interleaved)


def test_rope_copied_columns_keep_their_bits():
    q = torch.tensor([float("nan"), float("inf"), -0.0, 1e-40], dtype=torch.float32).repeat(16).to(BF).view(1, 1, 1, 64)
    f = freqs(8)
    for il in (False, True):
        y, _ = fa().fa_rope(q.to(DEV), inv_freq=f.to(DEV), interleaved=il)
        assert torch.equal(y.cpu().view(torch.int16)[..., 8:], q.view(torch.int16)[..., 8:])


def test_rope_empty():
    f = freqs(64).to(DEV)
    for shape in ((0, 5, 2, 64), (2, 0, 2, 64)):
        q = torch.zeros(shape, dtype=BF, device=DEV)
        assert fa().fa_rope(q, q, inv_freq=f)[0].shape == shape


def test_rope_inverse_gives_the_gradients_of_attention():
    """A training layer: rope, fa_fwd, fa_bwd, inverse rope; dq and dk of the
    unrotated inputs against the oracle's, formula and differences."""
    from oracle import attention as A
    from oracle import backward as B
    g = gen(11)
    q, k, v, dout = rnd(g, 1, 140, 4, 64), rnd(g, 1, 140, 2, 64), rnd(g, 1, 140, 2, 64), rnd(g, 1, 140, 4, 64)
    f = freqs(32)
    m = fa()
    fd = f.to(DEV)
    qr, kr = m.fa_rope(q.to(DEV), k.to(DEV), inv_freq=fd)
    out, lse, _ = m.fa_fwd(qr, kr, v.to(DEV), causal=True)
    dqr, dkr, dv, _ = m.fa_bwd(qr, kr, v.to(DEV), out, lse, dout.to(DEV), causal=True)
    dq, dk = m.fa_rope(dqr, dkr, inv_freq=fd, inverse=True)
    pos = np.arange(140)[None]
    rq, rk = R.rope(q, pos, f), R.rope(k, pos, f)
    tq, tk = torch.from_numpy(rq), torch.from_numpy(rk)
    gq, gk, gv = B.attention_grad(tq, tk, v, dout, causal=True)
    gq, gk = R.rope(gq, pos, f, inverse=True), R.rope(gk, pos, f, inverse=True)
    for got, ref in ((dq, gq), (dk, gk), (dv, gv)):
        got = got.double().cpu().numpy()
        # the backward's own bounds (relative L1 1e-2, cosine 0.9995)
        assert np.abs(got - ref).sum() <= 1e-2 * np.abs(ref).sum()
        assert (got * ref).sum() >= 0.9995 * np.linalg.norm(got) * np.linalg.norm(ref)

    def loss(qx, kx):
        o, _ = A.attention(R.rope(qx, pos, f), R.rope(kx, pos, f), v, causal=True)
        return (o * dout.double().numpy()).sum()
    q64, k64 = q.double().numpy(), k.double().numpy()
    for at in [(0, 100, 1, 3), (0, 139, 3, 20), (0, 50, 0, 40)]:
        e = np.zeros_like(q64)
        e[at] = 1e-4
        assert np.isclose((loss(q64 + e, k64) - loss(q64 - e, k64)) / 2e-4, gq[at], rtol=1e-4, atol=1e-7)
    e = np.zeros_like(k64)
    e[0, 60, 1, 17] = 1e-4
    assert np.isclose((loss(q64, k64 + e) - loss(q64, k64 - e)) / 2e-4, gk[0, 60, 1, 17], rtol=1e-4, atol=1e-7)


# ---- append ----

def cache_case(seed, lens, q_lens, hkv=2, d=128, page=16, hq=0, dtype=BF, extra_rows=(0, 0)):
    """A cache full of NaN, tables for the rows the append fills, packed new
    rows with ``extra_rows`` rows of no sequence before and after them."""
    g = gen(seed)
    n = len(lens)
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + extra_rows[0]
    total = int(cu[-1]) + extra_rows[1]
    kn, vn = rnd(g, total, hkv, d, dtype=dtype), rnd(g, total, hkv, d, dtype=dtype)
    q = rnd(g, total, hq, d, dtype=dtype) if hq else None
    if page:
        pages = [-(-(L + m) // page) for L, m in zip(lens, q_lens)]
        perm = torch.randperm(sum(pages) + 2, generator=g).to(torch.int32)
        bt = torch.full((n, max(1, max(pages))), -1, dtype=torch.int32)
        at = 0
        for s, m in enumerate(pages):
            bt[s, :m] = perm[at:at + m]
            at += m
        kc = torch.full((sum(pages) + 2, page, hkv, d), float("nan"), dtype=dtype)
    else:
        bt = None
        kc = torch.full((n, max(L + m for L, m in zip(lens, q_lens)) + 3, hkv, d), float("nan"), dtype=dtype)
    return dict(kn=kn, vn=vn, q=q, cu=torch.tensor(cu, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32),
                bt=bt, kc=kc, vc=kc.clone())


def run_append(c, f=None, check=True, **kw):
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    kc, vc = dev(c["kc"]), dev(c["vc"])
    q = dev(c["q"])
    q_out = None if q is None else torch.full_like(q, float("nan"))
    qo, lens, ws = fa().fa_kvcache_append(dev(c["kn"]), dev(c["vn"]), kc, vc, dev(c["lens"]), q=q, q_out=q_out,
                                          cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), inv_freq=dev(f),
                                          **{k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    torch.cuda.synchronize()
    if check:
        assert fa().fa_check_device_error(ws) == (0, 0)
    return qo, kc, vc, lens, ws


def check_append(c, f=None, **kw):
    qo, kc, vc, lens, _ = run_append(c, f, **kw)
    kw = {k: v for k, v in kw.items()}
    rq, rk, rv, rl = R.kvcache_append(c["kn"], c["vn"], c["kc"], c["vc"], c["lens"], q=c["q"], cu_seqlens_q=c["cu"],
                                      block_table=c["bt"], inv_freq=f, **kw)
    assert lens.cpu().tolist() == list(rl)
    il, m = kw.get("interleaved", False), kw.get("mscale", 1.0)
    # v: bit for bit, and rows nobody writes keep their NaN
    assert torch.equal(vc.cpu().view(torch.int16), torch.from_numpy(rv).to(vc.dtype).view(torch.int16))
    if f is None:
        assert torch.equal(kc.cpu().view(torch.int16), torch.from_numpy(rk).to(kc.dtype).view(torch.int16))
        if c["q"] is not None:
            there = ~np.isnan(rq[..., 0, 0])
            assert torch.equal(qo.cpu()[there], c["q"][there]) and torch.isnan(qo.cpu()[~there]).all()
        return
    # k: each written row against its rotation; the magnitudes of a row's pairs come from the unrotated append
    _, raw, _, _ = R.kvcache_append(c["kn"], c["vn"], c["kc"], c["vc"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"])
    there = ~np.isnan(rk[..., 0, 0])
    assert torch.isnan(kc.cpu()[torch.from_numpy(~there)]).all()
    sel = torch.from_numpy(there)
    assert_rotated(kc.cpu()[sel], rk[there], raw[there], f, m, il, "k")
    if c["q"] is not None:
        there = ~np.isnan(rq[..., 0, 0])
        sel = torch.from_numpy(there)
        assert torch.isnan(qo.cpu()[~sel]).all()
        assert_rotated(qo.cpu()[sel], rq[there], c["q"][sel], f, m, il, "q")


@pytest.mark.parametrize("page", [None, 1, 5, 16, 64, 256])
@pytest.mark.parametrize("rot,interleaved,dtype,d", [(128, False, BF, 128), (32, True, H, 64), (42, False, BF, 128), (0, False, H, 64)])
def test_append(page, rot, interleaved, dtype, d):
    c = cache_case(rot + (page or 0), [0, 3, 700, 16, 31], [4, 1, 33, 0, 17], d=d, page=page, hq=6, dtype=dtype, extra_rows=(2, 3))
    if page is None:
        c["kc"] = c["kc"][:, :740].contiguous()
        c["vc"] = c["vc"][:, :740].contiguous()
    f = freqs(rot) if rot else None
    check_append(c, f, interleaved=interleaved, mscale=1.2) if rot else check_append(c)


@pytest.mark.parametrize("n_seq", [1, 32, 33, 1000, 5000])
def test_append_finds_the_sequence_of_each_row(n_seq):
    rng = np.random.default_rng(n_seq)
    q_lens = rng.integers(0, 4, n_seq).tolist()
    q_lens[-1] = 2
    c = cache_case(n_seq, rng.integers(0, 20, n_seq).tolist(), q_lens, hkv=1, d=64, page=8)
    check_append(c, freqs(16))


def test_append_without_q_and_with_positions():
    c = cache_case(7, [5, 40], [9, 3])
    check_append(c, freqs(64))
    pos = torch.randint(0, 100000, (12,), generator=gen(8), dtype=torch.int32)
    check_append(c, freqs(64), positions=pos)


def test_append_fixed_length_rows():
    c = cache_case(9, [0, 20, 15], [4, 4, 4], hq=4, page=16)
    n, S = 3, 4
    c4 = dict(c, kn=c["kn"].view(n, S, 2, 128), vn=c["vn"].view(n, S, 2, 128), q=c["q"].view(n, S, 4, 128), cu=None)
    pos = torch.randint(0, 1000, (n, S), generator=gen(1), dtype=torch.int32)
    f = freqs(128)
    for kw in ({}, dict(positions=pos)):
        check_append(c4, f, **kw)


def test_append_of_nothing_writes_the_lengths():
    c = cache_case(10, [3, 0], [0, 0], extra_rows=(0, 2))
    check_append(c, freqs(64))
    c = cache_case(10, [3, 0], [0, 0])
    check_append(c, freqs(64))


def test_append_equals_the_append_of_the_attention_call():
    """Without rotation the cache after the call is that of fa_fwd_kvcache(append=True)."""
    c = cache_case(12, [30, 0, 100], [3, 8, 1], hq=4)
    c["kc"], c["vc"] = rnd(gen(1), *c["kc"].shape), rnd(gen(2), *c["vc"].shape)
    _, kc, vc, _, _ = run_append(c)
    k2, v2 = c["kc"].to(DEV), c["vc"].to(DEV)
    fa().fa_fwd_kvcache(c["q"].to(DEV), k2, v2, c["kn"].to(DEV), c["vn"].to(DEV), c["lens"].to(DEV), append=True,
                        cu_seqlens_q=c["cu"].to(DEV), block_table=c["bt"].to(DEV), max_seqlen_q=8, max_seqlen_k=101)
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_append_records_what_does_not_fit():
    m = fa()
    BOUNDS = m._lib.FA_ERR_DEVICE_BOUNDS
    # sequence 1 runs past its table, sequence 2 has a negative length: neither is read or written
    c = cache_case(13, [5, 10, 3], [4, 4, 4], hq=2)
    c["lens"] = torch.tensor([5, 16 * c["bt"].shape[1] - 3, -1], dtype=torch.int32)
    qo, kc, vc, lens, ws = run_append(c, freqs(64), check=False)
    rc, info = m.fa_check_device_error(ws)
    assert rc == BOUNDS and info in (1, 2)
    assert m.fa_check_device_error(ws)[0] == 0  # read and cleared
    assert lens.tolist() == [9, int(c["lens"][1]), -1]
    assert torch.isfinite(qo[:4]).all() and torch.isnan(qo[4:]).all()
    assert int(torch.isfinite(vc).all(-1).all(-1).sum()) == 4
    # a page outside the cache: that row alone is skipped
    c = cache_case(14, [15, 0], [3, 2], hq=2)
    c["bt"][0, 1] = c["kc"].shape[0]
    qo, kc, vc, lens, ws = run_append(c, freqs(64), check=False)
    assert m.fa_check_device_error(ws) == (BOUNDS, c["kc"].shape[0])
    assert lens.tolist() == [18, 2] and torch.isfinite(qo).all()
    assert int(torch.isfinite(vc).all(-1).all(-1).sum()) == 3
    # rows outside the packed tensor, a length below zero
    c = cache_case(15, [0, 0, 0], [2, 2, 2])
    c["cu"] = torch.tensor([0, 4, 2, 9], dtype=torch.int32)
    qo, kc, vc, lens, ws = run_append(c, freqs(64), check=False)
    assert m.fa_check_device_error(ws)[0] == BOUNDS
    assert lens.tolist() == [4, 0, 0]


def test_append_strided_rows_and_cache():
    """k, v, q slices of one fused projection; the cache with room between its heads' rows."""
    g = gen(16)
    fused = rnd(g, 9, 4 + 2 + 2, 64)
    c = cache_case(17, [3, 30], [5, 4], d=64, page=8)
    big_k, big_v = [torch.full((*c["kc"].shape[:3], 72), float("nan"), dtype=BF).to(DEV) for _ in range(2)]
    f = freqs(64)
    dev = fused.to(DEV)
    q_out = dev[:, :4]
    m = fa()
    _, lens, ws = m.fa_kvcache_append(dev[:, 4:6], dev[:, 6:], big_k[..., :64], big_v[..., :64], c["lens"].to(DEV), q=dev[:, :4],
                                      q_out=q_out, cu_seqlens_q=c["cu"].to(DEV), block_table=c["bt"].to(DEV), inv_freq=f.to(DEV))
    rq, rk, rv, _ = R.kvcache_append(fused[:, 4:6], fused[:, 6:], c["kc"], c["vc"], c["lens"], q=fused[:, :4], cu_seqlens_q=c["cu"],
                                     block_table=c["bt"], inv_freq=f)
    assert_rotated(dev[:, :4], rq, fused[:, :4], f, 1.0, False)
    assert torch.equal(dev[:, 4:].cpu(), fused[:, 4:])
    assert torch.equal(big_v[..., :64].cpu().view(torch.int16), torch.from_numpy(rv).to(BF).view(torch.int16))
    assert torch.isnan(big_v[..., 64:]).all() and torch.isnan(big_k[..., 64:]).all()
    assert m.fa_check_device_error(ws)[0] == 0


def test_capture_and_other_stream():
    """Both calls captured in a graph and replayed on new inputs; a call on a
    stream that is not the current one."""
    m = fa()
    g = gen(18)
    c = cache_case(19, [20, 3], [2, 1], hq=4)
    f = freqs(128).to(DEV)
    st = {k: v.to(DEV) for k, v in c.items() if v is not None}
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens = torch.empty(2, dtype=torch.int32, device=DEV)
    qo = torch.empty_like(st["q"])

    def step():
        m.fa_kvcache_append(st["kn"], st["vn"], st["kc"], st["vc"], st["lens"], q=st["q"], q_out=qo, cu_seqlens_q=st["cu"],
                            block_table=st["bt"], inv_freq=f, seqlens_out=lens, workspace=ws)
        return m.fa_rope(st["q"].unsqueeze(0), inv_freq=f)[0]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    new_q = rnd(g, *c["q"].shape)
    st["q"].copy_(new_q)
    st["lens"].copy_(torch.tensor([21, 4], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [23, 5]
    pos = np.array([21, 22, 4])
    assert_rotated(qo, R.rope(new_q, pos, f.cpu()), new_q, f.cpu(), 1.0, False)
    assert_rotated(y[0], R.rope(new_q, np.arange(3), f.cpu()), new_q, f.cpu(), 1.0, False)
    # another stream's handle: the output is allocated for that stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z, _ = m.fa_rope(st["q"].unsqueeze(0), inv_freq=f, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(z, y)
