"""GPU tests of the operators on an 8-bit KV cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

from norm_util import NORM, assert_normed, pair_size
from oracle import q8 as Q
from oracle import qknorm as N
from oracle import rotary as R
from q8_util import (BF, DEV, E4, H, assert_close, cache, check, chunk_case, codes_of, dev, gen, on_device, oracle, rnd, run)
from rope_util import assert_rotated

pytestmark = pytest.mark.gpu


def fa():
    import masked_flash_attention_gb300 as m
    return m


def freqs(rot):
    return fa().fa_rope_inv_freq(rot)[0] if rot else None


# ---- append ----

def append_case(seed, lens, q_lens, hkv=2, d=128, page=16, block=16, hq=0, dtype=BF, extra_rows=(0, 0), spread=2.0, fixed=False):
    """A cache that holds `lens` keys, with room for the new ones; packed new rows with rows of no sequence around them."""
    c = cache(seed, [L + m for L, m in zip(lens, q_lens)], hkv, d, page, block, spread)
    # what the append has not yet written is NaN, and so are the scales of blocks that no old token has
    for s, (L, m) in enumerate(zip(lens, q_lens)):
        for j in range(L, L + m):
            pg, r = (int(c["bt"][s, j // page]), j % page) if page else (s, j)
            for n in "kv":
                c[n][pg, r] = np.nan
                if j % block == 0:
                    c[n + "_scale"][pg, r // block] = np.nan
    g = gen(seed + 1)
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + extra_rows[0]
    total = int(cu[-1]) + extra_rows[1]
    new = {n: rnd(g, total, h, d, dtype=dtype, spread=spread) for n, h in (("kn", hkv), ("vn", hkv), ("q", max(hq, 1)))}
    c.update(new, cu=torch.tensor(cu, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32))
    if not hq:
        c["q"] = None
    if fixed:
        for n in ("kn", "vn", "q"):
            c[n] = None if c[n] is None else c[n].view(len(lens), q_lens[0], *c[n].shape[1:])
        c["cu"] = None
    return c


def run_append(c, f=None, check=True, on=None, **kw):
    on = on_device(c) if on is None else on
    q = dev(c["q"])
    q_out = None if q is None else torch.full_like(q, float("nan"))
    qo, lens, ws = fa().fa_kvcache_append_q8(dev(c["kn"]), dev(c["vn"]), *on, dev(c["lens"]), q=q, q_out=q_out, cu_seqlens_q=dev(c["cu"]),
                                             block_table=dev(c["bt"]), inv_freq=dev(f), **{k: dev(v) for k, v in kw.items()})
    torch.cuda.synchronize()
    if check:
        assert fa().fa_check_device_error(ws) == (0, 0)
    return qo, on, lens, ws


def same(got, ref, name):
    """Bit for bit, a NaN for a NaN."""
    got = Q.values(got) if got.dtype == E4 else got.double().cpu().numpy()
    diff = ~((got == ref) | (np.isnan(got) & np.isnan(ref)))
    assert not diff.any(), f"{name}: {int(diff.sum())} differ, first {np.argwhere(diff)[0]}: {got[diff][0]} for {ref[diff][0]}"


def check_append(c, f=None, **kw):
    qo, on, lens, _ = run_append(c, f, **kw)
    r = Q.append(c["kn"], c["vn"], c["k"], c["v"], c["k_scale"], c["v_scale"], c["lens"], q=c["q"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                 inv_freq=f, **kw)
    assert lens.cpu().tolist() == list(r["lens"])
    same(on[1], r["v"], "v")
    same(on[3], r["v_scale"], "v's scales")
    il, m, eps = kw.get("interleaved", False), kw.get("mscale", 1.0), kw.get("eps")
    if f is None and not eps:
        same(on[0], r["k"], "k")
        same(on[2], r["k_scale"], "k's scales")
        if c["q"] is not None:
            there = ~np.isnan(r["q"][..., 0, 0])
            assert torch.equal(qo.cpu()[there], c["q"][there]) and torch.isnan(qo.cpu()[~there]).all()
        return
    # k's fp32 error, per row of the new tokens: of the pair's magnitude in the normalised or raw row
    half = 0 if f is None else len(f)
    raw = N.norm(c["kn"], kw.get("k_weight"), eps) if eps else c["kn"].double().numpy()
    size = pair_size(raw, half, il)
    size[..., :2 * half] *= abs(m)
    err = ((NORM if eps else 0.0) + 5e-7) * 1.01 * size
    scale, ref_scale = on[2].double().cpu().numpy(), r["k_scale"]
    block = c["k"].shape[1] // ref_scale.shape[1]
    page = c["k"].shape[1]
    touched = ~np.isnan(r["k_exact"])
    # scales: the oracle's, or a step beside it where the largest element is as near to the border as the error
    other = ~((scale == ref_scale) | (np.isnan(scale) & np.isnan(ref_scale)))
    wide = err.max(initial=0.0)
    for at in np.argwhere(other):
        b = slice(at[1] * block, (at[1] + 1) * block)
        top = np.nanmax(np.abs(r["k_exact"][at[0], b, at[2]])) * ref_scale[tuple(at)]
        edge = 448.0 * min(scale[tuple(at)], ref_scale[tuple(at)])
        assert abs(top - edge) <= wide, f"scale at {at}: {scale[tuple(at)]} for {ref_scale[tuple(at)]}"
    got = Q.values(on[0])
    full = np.repeat(np.where(other, np.nan, ref_scale), block, 1)[..., None]  # (blocks of another scale: by their values below)
    # the error of each cache row: its token's, none for tokens rounded again
    e = np.zeros(got.shape)
    lead = raw.shape[:-2]
    where = R.seq_of_rows(lead[0], c["cu"]) if c["cu"] is not None else [(s, i) for s in range(lead[0]) for i in range(lead[1])]
    for at, (s, i) in zip(np.ndindex(*lead), where):
        if s >= 0:
            j = int(c["lens"][s]) + i
            e[(s, j) if c["bt"] is None else (int(c["bt"][s, j // page]), j % page)] = err[at]
    with np.errstate(invalid="ignore"):
        y = r["k_exact"]
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) * (1 + 2.0 ** -20) + e / full
        bad = touched & ~np.isnan(full) & ~(np.abs(got - np.clip(y, -448, 448)) <= tol)
        # (an element that is not finite is NaN)
    assert not bad.any(), f"k: {int(bad.sum())}, first {np.argwhere(bad)[0]}: {got[bad][0]} for {y[bad][0]}"
    rest = ~touched & np.isfinite(full * np.ones_like(got))
    assert np.array_equal(got[rest], r["k"][rest], equal_nan=True)
    if c["q"] is not None:
        there = ~np.isnan(r["q"][..., 0, 0])
        assert torch.isnan(qo.cpu()[~there]).all()
        got_q, ref_q, x = qo.cpu()[there], r["q"][there], c["q"][there]
        if not eps:
            assert_rotated(got_q, ref_q, x, f, m, il, "q")
        else:
            mag = pair_size(N.norm(x, kw.get("q_weight"), eps), half, il)
            mag[..., :2 * half] *= abs(m)
            h = torch.finfo(got_q.dtype).eps / 2
            tol = h * np.abs(ref_q) + (NORM + 5e-7) * 1.01 * mag + (2.0 ** -25 if got_q.dtype == H else 0.0)
            assert (np.abs(got_q.double().numpy() - ref_q) <= tol).all()


@pytest.mark.parametrize("page,block", [(None, 16), (None, 64), (16, 16), (48, 16), (32, 32), (64, 64), (192, 64), (128, 128), (256, 128)])
@pytest.mark.parametrize("rot,interleaved,dtype,d", [(128, False, BF, 128), (32, True, H, 64), (42, False, BF, 128), (0, False, H, 64), (0, False, BF, 128)])
def test_append(page, block, rot, interleaved, dtype, d):
    c = append_case(rot + (page or 0) + block, [0, 3, 200, 16, 31, 127], [4, 1, 133, 0, 17, 1], d=d, page=page, block=block, hq=6, dtype=dtype,
                    extra_rows=(2, 3))
    check_append(c, freqs(rot), interleaved=interleaved, mscale=1.2) if rot else check_append(c)


@pytest.mark.parametrize("rot,interleaved,dtype,d,block", [(128, False, BF, 128, 16), (64, True, H, 64, 32), (24, False, H, 64, 64),
                                                           (42, False, BF, 128, 128), (0, False, BF, 128, 16)])
def test_append_normalises(rot, interleaved, dtype, d, block):
    g = gen(rot)
    c = append_case(rot + 1, [5, 0, 90], [3, 70, 1], d=d, page=block, block=block, hq=5, dtype=dtype, extra_rows=(1, 1))
    kw = dict(eps=1e-5, q_weight=1 + 0.3 * torch.randn(d, generator=g), k_weight=(1 + 0.3 * torch.randn(d, generator=g)).to(dtype))
    check_append(c, freqs(rot), interleaved=interleaved, **kw)
    check_append(c, freqs(rot), interleaved=interleaved, eps=0.5)


@pytest.mark.parametrize("n_seq", [1, 32, 33, 1000, 5000])
def test_append_finds_the_sequence_of_each_row(n_seq):
    rng = np.random.default_rng(n_seq)
    q_lens = rng.integers(0, 4, n_seq).tolist()
    q_lens[-1] = 2
    check_append(append_case(n_seq, rng.integers(0, 20, n_seq).tolist(), q_lens, hkv=1, d=64, page=16))


@pytest.mark.parametrize("rows,block", [(7000, 16), (9000, 32), (20000, 128)])  # runs of one row up to a whole block
def test_append_of_long_prompts(rows, block):
    q_lens = [rows // 2, 3, rows // 2 - 40, 0, 37]
    c = append_case(rows, [17, 0, 5, 9, 300], q_lens, hkv=1, d=64, page=block, block=block, hq=2)
    check_append(c, freqs(64))


def test_append_in_steps_and_growing_scales():
    """Tokens that enter a block one by one, each larger than those before it, and then smaller ones."""
    lens, on = torch.zeros(2, dtype=torch.int32), None
    c = append_case(3, [0, 0], [1, 1], page=32, block=16, spread=0.0)
    c["bt"] = torch.tensor([[1], [2]], dtype=torch.int32)
    on = on_device(c)
    state = {n: c[n] for n in ("k", "v", "k_scale", "v_scale")}
    for step in range(20):
        size = 2.0 ** (2 * step if step < 9 else 18 - step)
        g = gen(100 + step)
        kn, vn = rnd(g, 2, 2, 128) * size, rnd(g, 2, 2, 128) * size
        if step == 4:
            kn[0] = 0  # zeros alone leave the scale
        _, lens_out, ws = fa().fa_kvcache_append_q8(dev(kn), dev(vn), *on, dev(lens), cu_seqlens_q=torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV),
                                                    block_table=dev(c["bt"]))
        r = Q.append(kn, vn, state["k"], state["v"], state["k_scale"], state["v_scale"], lens, cu_seqlens_q=[0, 1, 2], block_table=c["bt"])
        state = {n: r[n] for n in state}
        for t, n in zip(on, ("k", "v", "k_scale", "v_scale")):
            same(t, state[n], f"{n} at step {step}")
        lens = lens_out.cpu()
    assert lens.tolist() == [20, 20] and fa().fa_check_device_error(ws) == (0, 0)


def test_append_of_odd_values():
    """Zeros, infinities, NaN, values beyond every scale and under the smallest."""
    c = append_case(4, [3, 0, 0, 0], [2, 1, 1, 2], d=64, page=16, spread=0.0, dtype=BF)
    for n in ("kn", "vn"):
        c[n][0, 0, 3], c[n][0, 1, 5], c[n][1, 0, 7] = float("inf"), float("nan"), -float("inf")
        c[n][2] = 0
        c[n][3] = 1e-30
        c[n][4, 0], c[n][4, 1] = 1e20, 448.0 * 2.0 ** 40
        c[n][5, 0, :32] = float("nan")
        c[n][5, 1] = 448.0 * 2.0 ** -40
    check_append(c)


def test_append_without_q_and_with_positions():
    c = append_case(7, [5, 40], [9, 3])
    check_append(c, freqs(64))
    check_append(c, freqs(64), positions=torch.randint(0, 100000, (12,), generator=gen(8), dtype=torch.int32))


def test_append_fixed_length_rows():
    c = append_case(9, [0, 20, 15], [4, 4, 4], hq=4, fixed=True)
    check_append(c, freqs(128))
    check_append(c, freqs(128), positions=torch.randint(0, 1000, (3, 4), generator=gen(1), dtype=torch.int32))


def test_append_of_nothing_writes_the_lengths():
    check_append(append_case(10, [3, 0], [0, 0], extra_rows=(0, 2)), freqs(64))
    check_append(append_case(10, [3, 0], [0, 0]), freqs(64))


def test_append_records_what_does_not_fit():
    m = fa()
    BOUNDS = m._lib.FA_ERR_DEVICE_BOUNDS
    # sequence 1 runs past its table, sequence 2 has a negative length: neither is read or written
    c = append_case(13, [5, 10, 3], [4, 4, 4], hq=2)
    c["lens"] = torch.tensor([5, 16 * c["bt"].shape[1] - 3, -1], dtype=torch.int32)
    qo, on, lens, ws = run_append(c, freqs(64), check=False)
    rc, info = m.fa_check_device_error(ws)
    assert rc == BOUNDS and info in (1, 2) and m.fa_check_device_error(ws)[0] == 0
    assert lens.tolist() == [9, int(c["lens"][1]), -1]
    assert torch.isfinite(qo[:4]).all() and torch.isnan(qo[4:]).all()
    changed = (~np.isnan(Q.values(on[1])) & np.isnan(c["v"])).all(-1).all(-1)
    assert changed.sum() == 4 and changed[int(c["bt"][0, 0]), 5:9].all()
    # a page outside the cache: its block's rows are skipped, q is not
    c = append_case(14, [15, 0], [3, 2], hq=2)
    c["bt"][0, 1] = c["k"].shape[0]
    qo, on, lens, ws = run_append(c, freqs(64), check=False)
    assert m.fa_check_device_error(ws) == (BOUNDS, c["k"].shape[0])
    assert lens.tolist() == [18, 2] and torch.isfinite(qo).all()
    assert (~np.isnan(Q.values(on[1])) & np.isnan(c["v"])).all(-1).all(-1).sum() == 3
    # rows outside the packed tensor, a length below zero
    c = append_case(15, [0, 0, 0], [2, 2, 2])
    c["cu"] = torch.tensor([0, 4, 2, 9], dtype=torch.int32)
    c["bt"][:] = torch.tensor([[0], [1], [2]], dtype=torch.int32)
    qo, on, lens, ws = run_append(c, freqs(64), check=False)
    assert m.fa_check_device_error(ws)[0] == BOUNDS and lens.tolist() == [4, 0, 0]


def test_append_strided_rows_and_cache():
    """k, v, q slices of one fused projection; codes with room between their heads' rows, scales head-major."""
    g = gen(16)
    fused = rnd(g, 9, 8, 64)
    c = append_case(17, [3, 30], [5, 4], d=64, page=32, block=16)
    c.update(kn=fused[:, 4:6], vn=fused[:, 6:])
    on = on_device(c)
    wide = [torch.full((*t.shape[:3], 80), 0x7f, dtype=torch.uint8, device=DEV).view(E4) for t in on[:2]]
    for w, t in zip(wide, on):
        w.view(torch.uint8)[..., :64] = t.view(torch.uint8)
    scales = [t.permute(2, 0, 1).contiguous().permute(1, 2, 0) for t in on[2:]]
    x = dev(fused)
    f = freqs(64)
    _, lens, ws = fa().fa_kvcache_append_q8(x[:, 4:6], x[:, 6:], wide[0][..., :64], wide[1][..., :64], *scales, dev(c["lens"]), q=x[:, :4],
                                            q_out=x[:, :4], cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), inv_freq=dev(f))
    r = Q.append(fused[:, 4:6], fused[:, 6:], c["k"], c["v"], c["k_scale"], c["v_scale"], c["lens"], q=fused[:, :4], cu_seqlens_q=c["cu"],
                 block_table=c["bt"], inv_freq=f)
    assert_rotated(x[:, :4], r["q"], fused[:, :4], f, 1.0, False)
    assert torch.equal(x[:, 4:].cpu(), fused[:, 4:]) and fa().fa_check_device_error(ws)[0] == 0
    same(wide[1][..., :64].contiguous(), r["v"], "v")
    same(scales[1].contiguous(), r["v_scale"], "scales")
    assert (wide[0].view(torch.uint8)[..., 64:] == 0x7f).all() and (wide[1].view(torch.uint8)[..., 64:] == 0x7f).all()


# ---- reading back ----

@pytest.mark.parametrize("page,block,d,hkv,dtype", [(16, 16, 128, 8, BF), (96, 32, 64, 3, H), (128, 128, 128, 1, H), (None, 64, 64, 5, BF)])
def test_read(page, block, d, hkv, dtype):
    lens = [33, 0, 1, 700, 128]
    c = cache(page or 1, lens, hkv, d, page, block, spread=2.0)
    on = on_device(c)
    cu = torch.tensor([2, 35, 35, 36, 736, 864], dtype=torch.int32)
    ko, vo = (torch.full((870, hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    a, b, ws = fa().fa_kvcache_read_q8(*on, cu_seqlens_k=dev(cu), block_table=dev(c["bt"]), k_out=ko, v_out=vo)
    assert a is ko and b is vo and fa().fa_check_device_error(ws) == (0, 0)
    k2, v2, _ = fa().fa_kvcache_read_q8(*on, dev(torch.tensor(lens, dtype=torch.int32)), block_table=dev(c["bt"]), max_seqlen_k=701, dtype=dtype)
    for n, packed, padded in (("k", ko, k2), ("v", vo, v2)):
        full = Q.dequantised(c[n], c[n + "_scale"])
        assert (packed[:2] == 7).all() and (packed[864:] == 7).all()
        for s, L in enumerate(lens):
            rows = full[c["bt"][s].numpy()[:-(-L // page)]].reshape(-1, hkv, d)[:L] if page else full[s, :L]
            ref = torch.from_numpy(rows).to(dtype)  # one rounding, of none in bf16
            assert dtype == H or np.array_equal(ref.double().numpy(), rows)
            assert torch.equal(packed[int(cu[s]):int(cu[s]) + L].cpu(), ref) and torch.equal(padded[s, :L].cpu(), ref)


def test_read_leaves_other_rows_and_records_errors():
    m = fa()
    c = cache(21, [20, 40], page=16)
    on, lens = on_device(c), torch.tensor([20, 40], dtype=torch.int32, device=DEV)
    ko, vo = (torch.full((2, 50, 2, 128), 7.0, dtype=BF, device=DEV) for _ in range(2))
    m.fa_kvcache_read_q8(*on, lens, block_table=dev(c["bt"]), k_out=ko, v_out=vo)
    assert (ko[0, 20:] == 7).all() and (vo[1, 40:] == 7).all() and not (ko[1, :40] == 7).all(-1).any()
    # too long for the output, for the table; below zero
    for bad in ([51, 40], [20, 49], [-1, 40]):
        ko.fill_(7)
        _, _, ws = m.fa_kvcache_read_q8(*on, torch.tensor(bad, dtype=torch.int32, device=DEV), block_table=dev(c["bt"]), k_out=ko, v_out=vo)
        rc, info = m.fa_check_device_error(ws)
        s = 0 if bad[0] != 20 else 1
        assert rc == m._lib.FA_ERR_DEVICE_BOUNDS and info == s and (ko[s] == 7).all() and not (ko[1 - s] == 7).all()
    bt = c["bt"].clone()
    bt[1, 1] = -5
    ko.fill_(7)
    _, _, ws = m.fa_kvcache_read_q8(*on, lens, block_table=dev(bt), k_out=ko, v_out=vo)
    assert m.fa_check_device_error(ws)[0] == m._lib.FA_ERR_DEVICE_BOUNDS
    assert (ko[1, 16:32] == 7).all() and not (ko[1, :16] == 7).all(-1).any() and not (ko[1, 32:40] == 7).all(-1).any()
    _, _, ws = m.fa_kvcache_read_q8(*on, cu_seqlens_k=torch.tensor([0, 30, 20], dtype=torch.int32, device=DEV), total_k=30, block_table=dev(c["bt"]))
    assert m.fa_check_device_error(ws)[0] == m._lib.FA_ERR_DEVICE_BOUNDS
    empty, _, _ = m.fa_kvcache_read_q8(*on, cu_seqlens_k=torch.zeros(3, dtype=torch.int32, device=DEV), total_k=0, block_table=dev(c["bt"]))
    assert empty.shape == (0, 2, 128)


# ---- attention ----

def test_one_token_one_block():
    check(chunk_case(1, [1], [1], hq=1, hkv=1, d=64))


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (32, 32), (64, 64), (128, 128), (256, 32), (None, 16), (None, 128)])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, H)])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_pages_and_blocks(page, block, d, dtype, most):
    q_lens = [min(most, n) for n in (33, 1, 5, 40)]
    check(chunk_case(block, q_lens, [300, 17, 5, 129], hq=8, d=d, page=page, block=block, dtype=dtype))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (8, 2), (5, 1), (12, 2), (14, 2), (16, 1), (32, 1), (40, 1), (22, 1), (34, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens", [[1, 1], [2, 4], [70, 9]])
def test_heads(hq, hkv, d, q_lens):
    check(chunk_case(hq, q_lens, [200, 131], hq=hq, hkv=hkv, d=d, page=32, dtype=H if d == 64 else BF))


MASKS = [dict(), dict(causal=False), dict(window_left=37), dict(window_left=0), dict(window_left=200, window_right=3),
         dict(causal=False, window_right=10), dict(causal=False, window_left=20, window_right=0), dict(softcap=15.0), dict(softcap=400.0),
         dict(window_left=130, softcap=8.0, scale=0.3), dict(window_left=37, sink_keys=4), dict(window_left=0, sink_keys=1),
         dict(window_left=10, sink_keys=150), dict(window_left=300, sink_keys=500), dict(sink_keys=7), dict(causal=False, window_left=5, sink_keys=129),
         dict(window_left=16, window_right=0, sink_keys=16, softcap=20.0)]


@pytest.mark.parametrize("i", range(len(MASKS)))
@pytest.mark.parametrize("d,q_lens", [(64, [1, 1, 1, 1]), (128, [1, 3, 2, 4]), (64, [50, 3, 140, 1]), (128, [130, 1, 17, 33])])
def test_masks(i, d, q_lens):
    check(chunk_case(i, q_lens, [700, 150, 140, 33], hq=4, hkv=2, d=d, page=32, dtype=BF if d == 64 else H, **MASKS[i]))


@pytest.mark.parametrize("params", [{}, dict(softcap=15.0), dict(causal=False, window_right=20), dict(window_left=50, sink_keys=3)])
@pytest.mark.parametrize("d,q_lens", [(64, [1, 2]), (128, [60, 5])])
def test_alibi(params, d, q_lens):
    slopes = torch.tensor([0.5, 0.25, 0.125, 1.0, 0.01, 0.3])
    check(chunk_case(3, q_lens, [300, 90], hq=6, hkv=2, d=d, page=16, alibi_slopes=slopes, **params))


@pytest.mark.parametrize("params", [{}, dict(window_left=100), dict(softcap=30.0), dict(window_left=20, sink_keys=30)])
@pytest.mark.parametrize("d,q_lens", [(64, [4, 4, 4]), (128, [90, 200, 7])])
def test_prefix(params, d, q_lens):
    pre = torch.tensor([50, 260, 0], dtype=torch.int32)
    check(chunk_case(4, q_lens, [250, 200, 30], hq=4, d=d, page=16, prefix_lens=pre, **params))


@pytest.mark.parametrize("q_lens,kv_lens", [([3, 5, 2], [0, 2, 1]), ([40, 60, 33], [0, 13, 1])])
def test_rows_without_keys(q_lens, kv_lens):
    c = chunk_case(5, q_lens, kv_lens, d=64)
    out, lse = check(c)
    assert (out[:q_lens[0]] == 0).all() and torch.isneginf(lse[:, :q_lens[0]]).all()
    check(chunk_case(6, q_lens, [max(k, 1) + 40 for k in kv_lens], causal=False, window_left=3, window_right=2))


@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 2), (12, 12), (1, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("params", [{}, dict(window_left=2000, sink_keys=5), dict(window_left=100, sink_keys=1)])
def test_long_caches_are_split(hq, hkv, d, params):
    c = chunk_case(hq, [1, 2, 1], [9000, 3333, 40], hq=hq, hkv=hkv, d=d, page=64, **params)
    rc, p = fa().fa_fwd_chunk_q8_plan(c["q"], *(t.cpu() for t in on_device(c)), c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                                      max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"], **params)
    assert rc == 0 and (p["n_splits"] > 1) == (params.get("window_left") != 100)  # (a window of three tiles stays whole)
    check(c)


def test_many_sequences_and_empty_ones():
    rng = np.random.default_rng(8)
    n = 700
    kv = rng.integers(0, 40, n).tolist()
    check(chunk_case(8, [min(k, int(m)) for k, m in zip(kv, rng.integers(0, 3, n))], kv, hq=2, hkv=1, d=64, page=16))


@pytest.mark.parametrize("q_lens", [[1, 3], [40, 70]])
def test_scales_far_apart(q_lens):
    """Blocks of V 2^20 and more above others, and blocks of zeros: each weighs by its own keys."""
    c = chunk_case(9, q_lens, [300, 200], d=64, page=16)
    rng = np.random.default_rng(9)
    for n, hi in (("k", 2), ("v", 14)):
        c[n + "_scale"] = c[n + "_scale"] * 2.0 ** rng.integers(-hi, hi, c[n + "_scale"].shape)
    for s, j in ((0, 3), (1, 2)):
        pg = int(c["bt"][s, j])
        c["v"][pg], c["v_scale"][pg] = 0.0, 2.0 ** -40
        c["k"][int(c["bt"][s, j + 1])], c["k_scale"][int(c["bt"][s, j + 1])] = 0.0, 2.0 ** -40
    # weights of keys in small blocks next to large ones lie under 2^-14 of the top: counted by v_max
    check(c)


def test_extreme_scales():
    """V's scales at both ends of their range, with equal logits: the row sums hold both."""
    c = chunk_case(10, [1], [32], hq=1, hkv=1, d=64, page=16)
    c["q"].zero_()
    a, b = int(c["bt"][0, 0]), int(c["bt"][0, 1])
    c["v_scale"][a], c["v_scale"][b] = 2.0 ** 40, 2.0 ** -40
    out, lse = check(c)
    assert abs(float(lse[0, 0]) - np.log(32)) < 1e-5


@pytest.mark.parametrize("dtype", [BF, H])
@pytest.mark.parametrize("q_lens", [[2, 3], [60, 33]])
def test_sizes_of_queries(dtype, q_lens):
    """Rows of Q that are zero, tiny, large, or hold one large element."""
    c = chunk_case(11, q_lens, [100, 90], dtype=dtype)
    q = c["q"].float()
    q[0] = 0
    q[1] *= 1e-6
    q[2] *= 50
    q[3, :, 5] = 1000.0
    c["q"] = q.to(dtype)
    check(c)


@pytest.mark.parametrize("q_len", [5, 40])
def test_fixed_length_queries_and_padded_cache(q_len):
    check(chunk_case(12, [q_len] * 3, [q_len, 90, 200], hq=8, fixed=True, page=None, block=64))
    check(chunk_case(13, [q_len] * 3, [q_len, 90, 200], hq=8, fixed=True, page=48, d=64, dtype=H, window_left=60, sink_keys=9))


@pytest.mark.parametrize("q_lens", [[3, 1], [40, 20]])
def test_strides_and_untouched_rows(q_lens):
    c = chunk_case(14, q_lens, [100, 140], hq=8, d=64, extra=(3, 4))
    ref = oracle(c)
    out, lse, _ = run(c, fill=7.0)
    n = sum(q_lens)
    assert (out[:3] == 7).all() and (out[3 + n:] == 7).all() and (lse[:, :3] == 7).all() and (lse[:, 3 + n:] == 7).all()
    assert_close(c, out, lse, ref)
    # q and out inside wider rows, lse transposed, codes with room after each row, scales head-major
    m = fa()
    q = torch.zeros(c["q"].shape[0], 10, 72, dtype=BF, device=DEV)
    q[:, 1:9, :64] = dev(c["q"])
    o = torch.full_like(q, 7.0)
    l = torch.full((q.shape[0], 8), 7.0, device=DEV)
    on = on_device(c)
    wide = [torch.full((*t.shape[:3], 96), 0x7f, dtype=torch.uint8, device=DEV).view(E4) for t in on[:2]]
    for w, t in zip(wide, on):
        w.view(torch.uint8)[..., 16:80] = t.view(torch.uint8)
    scales = [t.permute(2, 0, 1).contiguous().permute(1, 2, 0) for t in on[2:]]
    m.fa_fwd_chunk_q8(q[:, 1:9, :64], wide[0][..., 16:80], wide[1][..., 16:80], *scales, dev(c["lens"]), out=o[:, 1:9, :64], lse=l.T,
                      cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"])
    assert torch.equal(o[3:3 + n, 1:9, :64], out[3:3 + n]) and torch.equal(l.T[:, 3:3 + n], lse[:, 3:3 + n])
    assert (o[:, 0] == 7).all() and (o[:, 9] == 7).all() and (o[..., 64:] == 7).all()


@pytest.mark.parametrize("q_lens", [[1, 4], [130, 9]])
def test_same_bits_again_and_without_skipping(q_lens):
    c = chunk_case(15, q_lens, [900, 300], window_left=100, sink_keys=20)
    a, b = run(c), run(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out, lse, _ = run(c, debug_flags=fa().FA_DEBUG_NO_SKIP)
    assert_close(c, out, lse, oracle(c))


@pytest.mark.parametrize("q_lens,d", [([1, 2, 1], 64), ([60, 20, 33], 128)])
def test_hidden_pages_are_not_read(q_lens, d):
    """Pages that the window hides from every row may be gone: their table entries hold anything."""
    c = chunk_case(16, q_lens, [900, 700, 800], hq=4, d=d, page=16, window_left=50, sink_keys=3)
    ref = oracle(c)
    for s, (n, L) in enumerate(zip(q_lens, (900, 700, 800))):
        c["bt"][s, 1:(L - n - 50) // 16] = 10**6
    out, lse, _ = run(c)
    assert_close(c, out, lse, ref)


@pytest.mark.parametrize("q_lens", [[1, 1], [3, 2], [50, 40]])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_rows_that_see_it(q_lens, d):
    """NaN codes in K and V of keys that only some rows see."""
    c = chunk_case(17, q_lens, [100, 90], hq=4, hkv=2, d=d, page=16, window_left=70)
    # V of a key behind the window of the last rows, and of the last key (seen by the last row alone); K of another sequence's last key
    for s, (n, L) in enumerate(zip(q_lens, (100, 90))):
        for j, h, col in ((L - n - 70, 0, 5), (L - 1, 1, 17)):
            c["v"][int(c["bt"][s, j // 16]), j % 16, h, col] = np.nan
    ro, rl, mass, size = ref = oracle(c)
    assert np.isnan(ro).any() and not np.isnan(mass).any()
    out, lse, _ = run(c)
    assert_close(c, out, lse, ref)
    # a NaN in K: the rows that see it are NaN whole, LSE too; the others stay
    c = chunk_case(18, q_lens, [100, 90], hq=4, hkv=2, d=d, page=16)
    clean = oracle(c)
    j = 99
    c["k"][int(c["bt"][0, j // 16]), j % 16, 1, 3] = np.nan
    out, lse, _ = run(c)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool)
    hit[q_lens[0] - 1, 2:] = True
    assert torch.isnan(out.cpu()[hit]).all() and torch.isnan(lse.T.cpu()[hit]).all()
    assert not torch.isnan(out.cpu()[~hit]).any() and not torch.isnan(lse.T.cpu()[~hit]).any()
    ro, rl, mass, size = clean
    keep = hit.numpy()
    assert_close({**c, "v": c["v"]}, torch.where(hit[..., None], torch.from_numpy(ro).to(out.dtype), out.cpu()),
                 torch.where(hit.T, torch.from_numpy(rl).float(), lse.cpu()), clean)
    assert keep.sum() == 2


def test_lengths_and_pages_that_do_not_fit():
    m = fa()
    BOUNDS = m._lib.FA_ERR_DEVICE_BOUNDS
    for q_lens in ([3, 2, 1], [50, 40, 60]):
        c = chunk_case(19, q_lens, [100, 60, 90])
        good, gl, _ = run(c)
        cu = c["cu"].tolist()
        for s, wrong in ((0, 101), (1, -1)):
            d = dict(c, lens=c["lens"].clone())
            d["lens"][s] = wrong
            out, lse, ws = run(d, check=False, fill=7.0)
            assert m.fa_check_device_error(ws) == (BOUNDS, s)
            for t in range(3):
                rows = slice(cu[t], cu[t + 1])
                if t == s:
                    assert (out[rows] == 7).all() and (lse[:, rows] == 7).all()
                else:
                    assert torch.equal(out[rows], good[rows]) and torch.equal(lse[:, rows], gl[:, rows])
        d = dict(c, bt=c["bt"].clone())
        d["bt"][1, 2] = c["k"].shape[0]
        out, lse, ws = run(d, check=False)
        assert m.fa_check_device_error(ws) == (BOUNDS, c["k"].shape[0])
        assert torch.equal(out[:cu[1]], good[:cu[1]]) and torch.equal(out[cu[2]:], good[cu[2]:])
        d = dict(c, max_q=q_lens[0] - 1)
        out, lse, ws = run(d, check=False, fill=7.0)
        assert m.fa_check_device_error(ws)[0] == BOUNDS and (out[:cu[1]] == 7).all()


def test_far_pages():
    """Offsets past 32 bits in the cache."""
    m = fa()
    n = 2**32 // (64 * 8 * 128) + 9
    kc = torch.empty(n, 64, 8, 128, dtype=torch.uint8, device=DEV).view(E4)
    vc = torch.empty(n, 64, 8, 128, dtype=torch.uint8, device=DEV).view(E4)
    ks, vs = (torch.ones(n, 4, 8, device=DEV) for _ in range(2))
    bt = torch.tensor([[n - 1, 3], [0, n - 2]], dtype=torch.int32)
    g = gen(20)
    kn, vn, q = rnd(g, 150, 8, 128), rnd(g, 150, 8, 128), rnd(g, 150, 16, 128)
    cu, past = torch.tensor([0, 80, 150], dtype=torch.int32), torch.zeros(2, dtype=torch.int32, device=DEV)
    _, lens, ws = m.fa_kvcache_append_q8(dev(kn), dev(vn), kc, vc, ks, vs, past, cu_seqlens_q=dev(cu), block_table=dev(bt))
    out, lse, ws2 = m.fa_fwd_chunk_q8(dev(q), kc, vc, ks, vs, lens, cu_seqlens_q=dev(cu), block_table=dev(bt), max_seqlen_q=80, max_seqlen_k=128)
    k, v, ws3 = m.fa_kvcache_read_q8(kc, vc, ks, vs, cu_seqlens_k=dev(cu), total_k=150, block_table=dev(bt))
    assert all(m.fa_check_device_error(w) == (0, 0) for w in (ws, ws2, ws3))
    small = dict(k=np.zeros((4, 64, 8, 128)), k_scale=np.ones((4, 4, 8)))
    r = Q.append(kn, vn, small["k"], small["k"], small["k_scale"], small["k_scale"], [0, 0], cu_seqlens_q=cu,
                 block_table=torch.tensor([[3, 1], [0, 2]]))
    c = dict(q=q, k=r["k"], v=r["v"], k_scale=r["k_scale"], v_scale=r["v_scale"], cu=cu, lens=lens.cpu(), bt=torch.tensor([[3, 1], [0, 2]]),
             max_k=128, params={})
    assert_close(c, out, lse, oracle(c))
    for t, name in ((k, "k"), (v, "v")):
        full = Q.dequantised(r[name], r[name + "_scale"])
        ref = np.concatenate([np.concatenate([full[3], full[1]])[:80], np.concatenate([full[0], full[2]])[:70]])
        assert np.array_equal(t.double().cpu().numpy(), ref)


@pytest.mark.parametrize("d,dtype,norm", [(128, BF, True), (64, H, False)])
def test_serving_steps(d, dtype, norm):
    """Prompts and then single tokens: normalised, rotated, quantised, attended to, with a window and sinks, as a
    server would; each step's cache against the oracle's append, its output against attention over that cache, and
    the same output from fa_fwd_chunk over the cache read back."""
    m = fa()
    g = gen(22)
    hq, hkv, page, block, n = 8, 2, 64, 32, 3
    f = freqs(d)
    bt = torch.randperm(12, generator=g).to(torch.int32).view(n, 4)
    c = dict(k=np.full((12, page, hkv, d), np.nan), v=np.full((12, page, hkv, d), np.nan), k_scale=np.full((12, 2, hkv), np.nan),
             v_scale=np.full((12, 2, hkv), np.nan), bt=bt)
    on = on_device(c)
    weights = dict(q_weight=1 + 0.2 * torch.randn(d, generator=g), k_weight=1 + 0.2 * torch.randn(d, generator=g), eps=1e-6) if norm else {}
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    for step, q_lens in enumerate([[100, 37, 1], [1, 1, 90], [1, 1, 1], [1, 0, 1], [30, 2, 1], [1, 1, 1]]):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
        total = int(cu[-1])
        q, k, v = rnd(g, total, hq, d, dtype=dtype), rnd(g, total, hkv, d, dtype=dtype), rnd(g, total, hkv, d, dtype=dtype)
        before = lens.cpu()
        held = dict(zip(("k", "v", "k_scale", "v_scale"), (Q.values(on[0]), Q.values(on[1]), on[2].double().cpu().numpy(), on[3].double().cpu().numpy())))
        qr, lens, _ = m.fa_kvcache_append_q8(dev(k), dev(v), *on, lens, q=dev(q), cu_seqlens_q=dev(cu), block_table=dev(bt), inv_freq=dev(f),
                                             workspace=ws, **{a: dev(b) for a, b in weights.items()})
        kw = dict(cu_seqlens_q=dev(cu), block_table=dev(bt), max_seqlen_q=max(q_lens), max_seqlen_k=256)
        out, lse, _ = m.fa_fwd_chunk_q8(qr, *on, lens, window_left=60, sink_keys=4, workspace=ws, **kw)
        plain, plain_lse, _ = m.fa_fwd_chunk_q8(qr, *on, lens, workspace=ws, **kw)
        back_k, back_v = (torch.zeros(n, 256, hkv, d, dtype=dtype, device=DEV) for _ in range(2))
        m.fa_kvcache_read_q8(*on, lens, block_table=dev(bt), k_out=back_k, v_out=back_v, workspace=ws)
        other, other_lse, _ = m.fa_fwd_chunk(qr, back_k, back_v, lens, cu_seqlens_q=dev(cu), max_seqlen_q=max(q_lens), max_seqlen_k=256)
        assert m.fa_check_device_error(ws) == (0, 0)
        r = Q.append(k, v, held["k"], held["v"], held["k_scale"], held["v_scale"], before, q=q, cu_seqlens_q=cu, block_table=bt, inv_freq=f, **weights)
        same(on[1], r["v"], f"v at step {step}")
        same(on[3], r["v_scale"], f"v's scales at step {step}")
        after = dict(q=qr.cpu(), k=Q.values(on[0]), v=Q.values(on[1]), k_scale=on[2].double().cpu().numpy(), v_scale=on[3].double().cpu().numpy(),
                     cu=cu, lens=lens.cpu(), bt=bt, max_k=256, params={})
        # a code is the oracle's or the next one where fp32 met a border: few are
        there = ~np.isnan(r["k"])
        assert (np.isnan(after["k"]) == ~there).all() and np.array_equal(after["k_scale"], r["k_scale"], equal_nan=True)
        off = there & (after["k"] != r["k"])
        assert off.sum() <= 1e-4 * there.sum() + 2
        assert (np.abs(after["k"] - r["k"])[off] <= np.maximum(2.0 ** -3 * np.abs(r["k"]), 2.0 ** -9)[off]).all()
        assert_close(after, out, lse, oracle(after, window_left=60, sink_keys=4), f"step {step}", window_left=60, sink_keys=4)
        ref = oracle(after)
        assert_close(after, plain, plain_lse, ref, f"step {step}, without a window")
        # both round P and the output once
        h = torch.finfo(dtype).eps / 2
        tol = 2 * h * np.abs(ref[0]) + (h + 2.0 ** -11 + 4e-4) * 1.01 * ref[2] + 2.0 ** -24
        assert (np.abs(plain.double().cpu().numpy() - other.double().cpu().numpy()) <= tol).all()
        assert (plain_lse - other_lse).abs().nan_to_num(0).max() <= 1e-4


def test_capture_streams_and_changed_lengths():
    """A decoding step (append, attention, reading back) captured and replayed with other lengths and inputs; the same on another stream."""
    m = fa()
    c = append_case(23, [40, 300], [1, 1], hq=8, page=64, block=16)
    f = dev(freqs(128))
    on = on_device(c)
    st = {k: dev(c[k]) for k in ("kn", "vn", "q", "cu", "lens", "bt")}
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)

    def step(on, stream=None):
        qr, lens, _ = m.fa_kvcache_append_q8(st["kn"], st["vn"], *on, st["lens"], q=st["q"], cu_seqlens_q=st["cu"], block_table=st["bt"],
                                             inv_freq=f, workspace=ws, stream=stream)
        out, lse, _ = m.fa_fwd_chunk_q8(qr, *on, lens, cu_seqlens_q=st["cu"], block_table=st["bt"], max_seqlen_q=1, max_seqlen_k=320,
                                        window_left=100, sink_keys=2, workspace=ws, stream=stream)
        k, v, _ = m.fa_kvcache_read_q8(*on, lens, block_table=st["bt"], max_seqlen_k=320, workspace=ws, stream=stream,
                                       k_out=torch.zeros(2, 320, 2, 128, dtype=BF, device=DEV), v_out=torch.zeros(2, 320, 2, 128, dtype=BF, device=DEV))
        return qr, out, lse, k, v
    s = torch.cuda.Stream()
    warm = [t.clone() for t in on]
    with torch.cuda.stream(s):
        step(warm)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    mine = [t.clone() for t in on]
    with torch.cuda.graph(graph):
        got = step(mine)
    for t, x in zip(mine, on):
        t.copy_(x)
    st["lens"].copy_(torch.tensor([17, 250], dtype=torch.int32))
    st["q"].copy_(rnd(gen(24), *c["q"].shape))
    again = [t.clone() for t in on]
    graph.replay()
    torch.cuda.synchronize()
    now = step(again)
    assert all(torch.equal(a, b) for a, b in zip(got, now))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(mine, again))  # (NaN scales too)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step([t.clone() for t in again], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(other[1], now[1]) and m.fa_check_device_error(ws) == (0, 0)


def test_small_workspace_and_misaligned_arguments():
    m = fa()
    c = chunk_case(25, [1, 1], [5000, 9], page=64)
    on = on_device(c)
    call = lambda ws=None, q=None, on=on: m.fa_fwd_chunk_q8(dev(c["q"]) if q is None else q, *on, dev(c["lens"]), cu_seqlens_q=dev(c["cu"]),  # noqa: E731
                                                           block_table=dev(c["bt"]), max_seqlen_q=1, max_seqlen_k=5000, workspace=ws)
    rc, p = m.fa_fwd_chunk_q8_plan(dev(c["q"]), *on, dev(c["lens"]), cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), max_seqlen_q=1, max_seqlen_k=5000)
    assert rc == 0
    for bad in (p["workspace_bytes"] - 1, 255):
        with pytest.raises(m.FaError) as e:
            call(torch.zeros(bad, dtype=torch.uint8, device=DEV))
        assert e.value.status == m._lib.FA_ERR_WORKSPACE
    call(torch.zeros(p["workspace_bytes"], dtype=torch.uint8, device=DEV))
    flat = torch.zeros(on[0].numel() + 16, dtype=torch.uint8, device=DEV)[8:8 + on[0].numel()].view(E4).view(on[0].shape)
    for k in ((flat, *on[1:]), (on[0], on[1], on[2].cpu(), on[3]), (on[0].view(torch.uint8), *on[1:])):
        with pytest.raises(m.FaError):
            call(on=k)


def test_shared_and_repeated_pages():
    """Sequences that share their first pages, and a page that stands twice in a table."""
    c = chunk_case(26, [2, 3, 1], [100, 90, 120], page=16)
    c["bt"][1, :3] = c["bt"][0, :3]
    c["bt"][2, 4] = c["bt"][2, 1]
    check(c)


@pytest.mark.parametrize("q_lens", [[1, 2], [4, 30]])
def test_wait_that_runs_out_is_reported(q_lens):
    """The first copy of K is never sent (FA_DEBUG_WITHHOLD): the bounded waits give up, the
    status is reported, and the next call on the workspace is right."""
    m = fa()
    c = chunk_case(27, q_lens, [60, 200])
    _, _, ws = run(c, check=False, debug_flags=m.FA_DEBUG_WITHHOLD)
    assert m.fa_check_device_error(ws)[0] == m._lib.FA_ERR_DEVICE_TIMEOUT
    out, lse, _ = run(c, workspace=ws)
    assert_close(c, out, lse, oracle(c))


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 2], [5000, 60, 700]), ([300, 1, 90], [1500, 60, 700])])
def test_two_streams_at_once(q_lens, kv_lens):
    """Two steps on two streams, each with its own workspace, a few times over."""
    m = fa()
    cs = [chunk_case(28 + i, q_lens, kv_lens, hq=8, window_left=900 + i, sink_keys=3) for i in range(2)]
    on = [on_device(c) for c in cs]
    st = [{k: dev(c[k]) for k in ("q", "cu", "lens", "bt")} for c in cs]

    def step(i, stream=None):
        return m.fa_fwd_chunk_q8(st[i]["q"], *on[i], st[i]["lens"], cu_seqlens_q=st[i]["cu"], block_table=st[i]["bt"], max_seqlen_q=max(q_lens),
                                 max_seqlen_k=max(kv_lens), workspace=ws[i], stream=stream, **cs[i]["params"])[:2]
    ws = [torch.zeros(64 << 20, dtype=torch.uint8, device=DEV) for _ in cs]
    one = [[t.clone() for t in step(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [step(i, s.cuda_stream) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(one, got) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,hq,hkv,d", [(3000, 40, 3, 128), (900, 17, 8, 64), (6000, 9, 1, 64)])
def test_append_shares_of_warps(rows, hq, hkv, d):
    """q's heads in one share of rounds and in several, the last one not full; weights off a 16-byte boundary."""
    g = gen(rows)
    c = append_case(rows, [7, 0, 40], [rows // 2, 3, rows - rows // 2 - 3], hkv=hkv, d=d, page=32, block=32, hq=hq)
    w = (1 + 0.3 * torch.randn(2, d + 1, generator=g)).to(BF)
    qo, on, _, _ = run_append(c, freqs(d), eps=1e-5, q_weight=dev(w)[0, 1:], k_weight=dev(w)[1, 1:])
    qa, on2, _, _ = run_append(c, freqs(d), eps=1e-5, q_weight=w[0, 1:].clone(), k_weight=w[1, 1:].clone())
    assert torch.equal(qo, qa) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(on, on2))
    check_append(c, freqs(d), eps=1e-5, q_weight=w[0, 1:].clone(), k_weight=w[1, 1:].clone())


@pytest.mark.parametrize("n_seq", [1, 31, 33, 1100])
def test_read_finds_the_sequence_of_each_row(n_seq):
    """Short and empty sequences, packed, with rows of none before and behind."""
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 5, n_seq).tolist()
    lens[n_seq // 2] = 70
    c = cache(n_seq, lens, 1, 64, 16, 16)
    cu = np.concatenate([[0], np.cumsum(lens)]) + 3
    ko, vo = (torch.full((int(cu[-1]) + 40, 1, 64), 7.0, dtype=BF, device=DEV) for _ in range(2))
    _, _, ws = fa().fa_kvcache_read_q8(*on_device(c), cu_seqlens_k=dev(torch.tensor(cu, dtype=torch.int32)), block_table=dev(c["bt"]), k_out=ko, v_out=vo)
    assert fa().fa_check_device_error(ws) == (0, 0)
    for n, got in (("k", ko.cpu()), ("v", vo.cpu())):
        full = Q.dequantised(c[n], c[n + "_scale"])
        assert (got[:3] == 7).all() and (got[int(cu[-1]):] == 7).all()
        for s, L in enumerate(lens):
            rows = full[c["bt"][s].numpy()[:-(-L // 16)]].reshape(-1, 1, 64)[:L]
            assert np.array_equal(got[int(cu[s]):int(cu[s]) + L].double().numpy(), rows)


def test_nan_far_back_in_a_long_cache():
    """A NaN in V far back in a long cache reaches the rows that see it, with tiles that are seen whole before and behind it."""
    c = chunk_case(30, [300, 40], [3000, 1700], hq=4, hkv=1, page=64, block=32, window_left=1200)
    pg, r = int(c["bt"][0, 2000 // 64]), 2000 % 64
    c["v"][pg, r, 0, 5] = np.nan
    out, lse, _ = run(c)
    assert np.isfinite(lse.cpu().numpy()).all()
    i = np.arange(300) + 2700  # the positions of the first sequence's rows
    sees = (i >= 2000) & (i - 1200 <= 2000)
    got = torch.isnan(out[:300]).any(-1).all(-1).cpu().numpy()
    assert np.array_equal(got, sees) and sees.all()
    clean = dict(c, v=c["v"].copy())
    clean["v"][pg, r, 0, 5] = 0.0
    a, b, _ = run(clean)
    keep = torch.ones(128, dtype=torch.bool)
    keep[5] = False
    assert torch.isfinite(a).all() and torch.equal(a[..., keep.to(a.device)], out[..., keep.to(out.device)]) and torch.equal(b, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,params", [([1, 1, 2], [5000, 1300, 40], dict(window_left=1200, sink_keys=40)),
                                                   ([1, 1, 1], [5000, 1100, 1000], dict(window_left=900, causal=False, window_right=100)),
                                                   ([1, 4], [1400, 1407], {}), ([1] * 64, [2000 - 31 * i for i in range(64)], {})])
def test_units_that_stay_whole(d, q_lens, kv_lens, params):
    """Up to 16 tiles to a CTA, without a planner: whole caches, and windows far along them with and without first keys."""
    check(chunk_case(31, q_lens, kv_lens, d=d, **params))


@pytest.mark.parametrize("d,hkv,params", [(64, 3, {}), (128, 2, dict(window_left=70, sink_keys=9)), (128, 1, dict(softcap=20.0))])
def test_many_pieces_of_a_cta(d, hkv, params):
    """Many sequences of many rows, some without tokens or keys of their own before them: several pieces to each CTA, one behind another."""
    rng = np.random.default_rng(d + hkv)
    q = [0 if x < 3 else int(x) for x in rng.integers(0, 90, 500)]
    q[7] = 150
    kv = [n + int(x) for n, x in zip(q, rng.integers(0, 260, 500))]
    check(chunk_case(d + hkv, q, kv, hq=2 * hkv, hkv=hkv, d=d, page=32, block=32, **params))


def nan_tokens(c, s, js, quiet=None, scale=None):
    """V of keys js of sequence s all NaN; quiet: their K such that a q of ones times d has a logit of -7 d sqrt(1 / d)
    (-448 in a block of scale 2^-6); scale: that of V's blocks they stand in."""
    page, block = c["k"].shape[1], c["k"].shape[1] // c["k_scale"].shape[1]
    for j in js:
        pg, r = int(c["bt"][s, j // page]), j % page
        c["v"][pg, r] = np.nan
        if quiet:
            c["k"][pg, r], c["k_scale"][pg, r // block] = -448.0, 2.0 ** -6
        if scale:
            c["v_scale"][pg, r // block] = scale


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len,hq", [(1, 4), (3, 4), (3, 8), (40, 4)])
@pytest.mark.parametrize("kv_len", [1024, 1025, 1030, 161])
@pytest.mark.parametrize("which", ["last block", "last key"])
def test_nan_of_a_small_block_after_earlier_keys(d, q_len, hq, kv_len, which):
    """The newest tokens' V all NaN, as the append leaves a block that holds nothing else: scale 2^-40.  Its keys' weights,
    2^-34 and less of those of the blocks before it, still bring the NaN to the rows that see them, and to no others."""
    c = chunk_case(q_len + kv_len, [q_len, 1], [kv_len, 200], hq=hq, hkv=2, d=d, page=16)
    first = (kv_len - 1) // 16 * 16
    nan_tokens(c, 0, range(first if which == "last block" else kv_len - 1, kv_len), scale=2.0 ** -40)
    ro, rl, mass, size = ref = oracle(c)
    assert np.isnan(ro[q_len - 1]).all() and not np.isnan(ro[q_len]).any() and not np.isnan(mass).any()
    out, lse, _ = run(c)
    assert_close(c, out, lse, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len,hq", [(1, 4), (3, 4), (3, 8), (40, 4)])
@pytest.mark.parametrize("scale", [None, 1.0])
@pytest.mark.parametrize("at", [1028, 129, 31, 9])
def test_nan_of_a_key_of_no_weight(d, q_len, hq, scale, at):
    """A NaN whose key has a logit 56 to 896 below the others: weights under fp16's, and under those of fp32.  The rows that
    see the key are NaN, in runs of keys that all rows see and in those at both ends of a window."""
    c = chunk_case(at, [q_len], [1030], hq=hq, hkv=2, d=d, page=16, window_left=1030 - q_len - at if at < 100 else -1, scale=scale)
    c["q"] = torch.ones_like(c["q"])
    nan_tokens(c, 0, [at], quiet=True)
    ro, rl, mass, size = ref = oracle(c)
    sees = np.isnan(ro).all((1, 2))
    assert sees.any() and np.array_equal(sees, np.isnan(ro).any((1, 2))) and (q_len == 1 or not sees.all() or at == 129)
    out, lse, _ = run(c)
    assert_close(c, out, lse, ref)


def by_value(c, on, r, err):
    """K's codes times the scales that were written, of all blocks, whatever scale each came out with: the new tokens' and the
    old ones' values to half a step of that scale (a code: 2^-4 of it, at least 2^-10), and fp32's error of new ones."""
    page, shape = c["k"].shape[1], c["k"].shape
    block = page // c["k_scale"].shape[1]
    wide = lambda s: np.repeat(s, block, 1)[..., None]  # noqa: E731
    got, scale = Q.values(on[0]), on[2].double().cpu().numpy()
    was = c["k"] * wide(c["k_scale"])  # (the old tokens; NaN elsewhere)
    new = r["k_exact"] * wide(r["k_scale"])
    e, fresh = np.zeros(shape), np.zeros(shape, dtype=bool)
    lead = c["kn"].shape[:-2]
    for at, (s, i) in zip(np.ndindex(*lead), R.seq_of_rows(lead[0], c["cu"])):
        if s >= 0:
            j = int(c["lens"][s]) + i
            e[int(c["bt"][s, j // page]), j % page] = err[at]
            fresh[int(c["bt"][s, j // page]), j % page] = True
    ref = np.where(fresh, new, was)
    kept = ~np.isnan(ref)
    assert np.array_equal(kept, ~np.isnan(got)) and kept.any()
    with np.errstate(invalid="ignore"):
        tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide(scale)) * (1 + 2.0 ** -20) + e
        bad = kept & ~(np.abs(got * wide(scale) - ref) <= tol)
    assert not bad.any(), f"{int(bad.sum())}, first {np.argwhere(bad)[0]}"
    return scale


@pytest.mark.parametrize("n_new,d,dtype", [(1, 128, BF), (2, 64, H)])
def test_append_codes_where_a_scale_is_a_step_off(n_new, d, dtype):
    """Normalised rows whose every element is 448 but for fp32's error: the scale is 1, or 2 where that error carries an
    element past 448, and the codes are those of the scale that was written, the old tokens' among them."""
    g, n = gen(d), 300
    c = append_case(d, [5, 0, 16] * (n // 3), [n_new] * n, hkv=2, d=d, page=16, block=16, dtype=dtype, spread=0.0)
    rows = 1.0 + torch.rand(n * n_new, 2, 1, generator=g)
    c["kn"] = (rows * torch.sign(torch.randn(n * n_new, 2, d, generator=g) + 1e-3)).to(dtype)
    # old tokens at up to 448 times a scale of 1
    old = ~np.isnan(c["k_scale"])
    c["k_scale"] = np.where(old, 1.0, np.nan)
    w, eps = torch.full((d,), 448.0), 1e-12
    qo, on, lens, _ = run_append(c, None, eps=eps, k_weight=w)
    r = Q.append(c["kn"], c["vn"], c["k"], c["v"], c["k_scale"], c["v_scale"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                 k_weight=w, eps=eps)
    scale = by_value(c, on, r, NORM * np.abs(N.norm(c["kn"], w, eps)))
    there = ~np.isnan(r["k_scale"])
    assert (r["k_scale"][there] == 1).all() and np.isin(scale[there], (1.0, 2.0)).all()


@pytest.mark.parametrize("rot,interleaved,d,block,eps", [(128, False, 128, 16, 1e-5), (64, True, 64, 32, None), (42, False, 128, 64, 1e-5)])
def test_append_codes_by_value(rot, interleaved, d, block, eps):
    c = append_case(rot + 50, [5, 0, 90, 200], [300, 70, 1, 40], d=d, page=block, block=block, hq=2, extra_rows=(1, 1))
    f = freqs(rot)
    w = 1 + 0.3 * torch.randn(d, generator=gen(rot)) if eps else None
    qo, on, lens, _ = run_append(c, f, interleaved=interleaved, eps=eps, k_weight=w)
    r = Q.append(c["kn"], c["vn"], c["k"], c["v"], c["k_scale"], c["v_scale"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                 inv_freq=f, interleaved=interleaved, k_weight=w, eps=eps)
    raw = N.norm(c["kn"], w, eps) if eps else c["kn"].double().numpy()
    by_value(c, on, r, ((NORM if eps else 0.0) + 5e-7) * 1.01 * pair_size(raw, len(f), interleaved))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens", [[2, 3], [40, 33]])
def test_logits_under_the_range_of_fp32(d, q_lens):
    """Rows of Q of 1e-30 over keys of zeros (scale 2^-40), with a scale of 1e-6: all logits are 0, masks hold."""
    c = chunk_case(32, q_lens, [100, 90], d=d, page=16, scale=1e-6)
    c["q"] = c["q"] * 1e-30
    c["k"] = np.where(np.isnan(c["k"]), np.nan, 0.0)
    c["k_scale"] = np.where(np.isnan(c["k_scale"]), np.nan, 2.0 ** -40)
    check(c)
