"""GPU tests of fa_fwd_chunk against the fp64 oracle."""
import numpy as np
import pytest
import torch

from chunk_util import BF, DEV, H, assert_close, case, check, dev, oracle, rnd, run

pytestmark = pytest.mark.gpu


def fa():
    import masked_flash_attention_gb300 as m
    return m


def test_one_token_one_tile():
    check(case(0, [1], [100], hq=4, hkv=1, page=16))


@pytest.mark.parametrize("page", [16, 64, 128, 256, 24, 8, 5, 2, 1, None])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, H)])
def test_pages(page, d, dtype):
    """Lengths on, before and after the edges of tiles, pages and MMA steps; a
    sequence without new tokens, one without keys, one with a single key."""
    check(case(1, [3, 1, 0, 130, 2, 1, 17], [127, 128, 50, 129, 0, 1, 300], page=page, d=d, dtype=dtype, hq=6, hkv=2), f"page {page}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (8, 2), (5, 1), (12, 2), (14, 2), (32, 1), (40, 1), (64, 1), (130, 1), (22, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_heads(hq, hkv, d):
    check(case(2, [1, 33, 70], [200, 33, 310], hq=hq, hkv=hkv, d=d, dtype=H if hq % 2 else BF), f"{hq}/{hkv}")


@pytest.mark.parametrize("i,params", list(enumerate([
    dict(causal=False), dict(window_left=0), dict(window_left=100), dict(window_left=40, window_right=0, softcap=20.0),
    dict(causal=False, window_left=30, window_right=90), dict(causal=False, window_right=5), dict(softcap=30.0),
    dict(scale=0.3), dict(window_left=2**31 - 1, window_right=2**31 - 1)])))
@pytest.mark.parametrize("d", [64, 128])
def test_masks(i, params, d):
    check(case(10 + i, [40, 1, 200, 300], [400, 350, 200, 290], d=d, page=16), str(params), logits=4.0, **params)


@pytest.mark.parametrize("params", [{}, dict(softcap=15.0), dict(causal=False, window_right=20), dict(window_left=150)])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, H)])
def test_alibi(params, d, dtype):
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(6)])
    c = case(30, [64, 1, 150], [400, 500, 150], hq=6, hkv=2, d=d, dtype=dtype)
    out, lse, _ = run(c, alibi_slopes=slopes, **params)
    assert_close(out, lse, oracle(c, alibi_slopes=slopes, **params), str(params), logits=2.0, n_keys=500)


@pytest.mark.parametrize("params", [{}, dict(window_left=100), dict(softcap=30.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix(params, d):
    c = case(40, [50, 200, 1, 130, 90, 10], [300, 200, 129, 260, 90, 400], d=d, page=16)
    pre = torch.tensor([0, 150, 40, 260, 1000, 395], dtype=torch.int32)
    check(c, str(params), prefix_lens=pre, **params)


def test_rows_without_keys():
    """More rows than keys, and windows that leave some rows nothing: 0 and -inf
    there, and the other rows of the same tiles right."""
    c = case(50, [150, 40, 5], [20, 0, 3], d=128)
    out, lse = check(c)
    assert (out[:130] == 0).all() and torch.isneginf(lse[:, :130]).all()
    c = case(51, [30], [300], d=64)
    out, lse = check(c, causal=False, window_left=-1, window_right=0)
    c = case(52, [300], [130], d=64)
    check(c, causal=False, window_left=10)  # the last rows' windows end before the first row's begin
    check(c, window_left=10)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (64, 1, 1), (64, 12, 12)])
def test_long_caches_are_split(d, hq, hkv):
    """Few units over many key tiles: split along the keys and joined; long and
    short sequences side by side."""
    c = case(60, [1, 40, 7], [9000, 5000, 100], hq=hq, hkv=hkv, d=d, page=32)
    out, lse, ws = run(c)
    assert_close(out, lse, oracle(c), n_keys=9000)
    counts = ws[256:272].view(torch.int32).tolist()
    assert counts[2] > 0 and counts[1] >= 2 * counts[2], counts
    # a row none of whose keys lie in some pieces
    c = case(61, [3], [7000], hq=hq, hkv=hkv, d=d, page=32)
    check(c, window_left=300)
    check(c, causal=False, window_right=10)


def test_many_sequences_and_empty_ones():
    rng = np.random.default_rng(7)
    q_lens = rng.integers(0, 3, 3000).tolist()
    kv = rng.integers(0, 60, 3000).tolist()
    check(case(70, q_lens, kv, hq=2, hkv=1, d=64, page=8))


def test_large_logits():
    """Rows whose maxima grow by far more than 2^8 from tile to tile (the
    reference is raised and O rescaled), and fall again."""
    for d, dtype in ((128, BF), (64, H)):
        c = case(80, [70, 2], [600, 900], d=d, dtype=dtype)
        ramp = torch.linspace(0.05, 4.0, 16)
        bt = c["bt"]
        for s in range(2):
            for p in range(bt.shape[1]):
                if bt[s, p] >= 0:
                    c["kc"][int(bt[s, p])] *= ramp[p % 16].item()
        # scale 1 and keys up to 4 times as large: a logit is off by up to 128 * 6e-8 * 82 * 4 = 2.5e-3
        check(c, f"ramp {d}", logits=30.0, scale=1.0)


def test_fixed_length_queries_and_padded_cache():
    check(case(90, [9, 9, 9], [100, 9, 33], page=None, d=64, fixed=True))
    check(case(91, [130, 130], [300, 130], page=16, d=128, fixed=True))


def test_strides_and_untouched_rows():
    """q, out, LSE and cache as slices of wider tensors; rows of no sequence and
    the columns between stay as they were."""
    c = case(100, [5, 60], [80, 61], hq=4, hkv=2, d=64, page=8, extra=(3, 4))
    out, lse, _ = run(c, fill=7.0)
    ref = oracle(c)
    assert_close(out, lse, ref)
    assert (out[:3] == 7).all() and (out[-4:] == 7).all() and (lse[:, :3] == 7).all() and (lse[:, -4:] == 7).all()
    m = fa()
    wide_q = torch.full((72, 4 + 3, 64 + 16), float("nan"), dtype=BF, device=DEV)
    wide_q[:, :4, :64] = c["q"].to(DEV)
    wide_o = torch.full((72, 9, 64 + 8), 7.0, dtype=BF, device=DEV)
    wide_l = torch.full((72, 8), 7.0, device=DEV)
    n_pages, page = c["kc"].shape[:2]
    wide_c = torch.full((n_pages, 2, page, 2, 64), float("nan"), dtype=BF, device=DEV)  # k and v pages in one pool
    wide_c[:, 0], wide_c[:, 1] = c["kc"].to(DEV), c["vc"].to(DEV)
    o2, l2, ws = m.fa_fwd_chunk(wide_q[:, :4, :64], wide_c[:, 0], wide_c[:, 1], dev(c["lens"]), out=wide_o[:, 2:6, :64],
                                lse=wide_l[:, 1:5].T, cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), max_seqlen_q=60,
                                max_seqlen_k=80)
    assert m.fa_check_device_error(ws) == (0, 0)
    assert torch.equal(o2[3:68], out[3:68]) and torch.equal(l2[:, 3:68], lse[:, 3:68])
    assert (wide_o[:, :2] == 7).all() and (wide_o[:, 6:] == 7).all() and (wide_o[:, :, 64:] == 7).all() and (wide_o[:3] == 7).all()
    assert (wide_l[:, 0] == 7).all() and (wide_l[:, 5:] == 7).all()


def test_heads_major_cache():
    """A cache [pages, Hkv, page, d] seen as [pages, page, Hkv, d]."""
    c = case(101, [20, 1], [200, 77], d=128)
    out, lse, _ = run(c)
    c2 = dict(c)
    c2["kc"], c2["vc"] = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (c["kc"], c["vc"])]
    m = fa()
    o2, l2, _ = m.fa_fwd_chunk(dev(c["q"]), c["kc"].transpose(1, 2).contiguous().to(DEV).transpose(1, 2),
                               c["vc"].transpose(1, 2).contiguous().to(DEV).transpose(1, 2), dev(c["lens"]),
                               cu_seqlens_q=dev(c["cu"]), block_table=dev(c["bt"]), max_seqlen_q=20, max_seqlen_k=200)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_same_bits_again_and_without_skipping():
    m = fa()
    c = case(110, [1, 200, 40], [5000, 900, 1000], d=128)
    a = run(c)
    for _ in range(3):
        b = run(c, workspace=a[2])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # every tile scheduled as PARTIAL: other splits, the same values
    out, lse, _ = run(c, debug_flags=m.FA_DEBUG_NO_SKIP, window_left=500)
    assert_close(out, lse, oracle(c, window_left=500), n_keys=5000)


def test_lengths_and_pages_that_do_not_fit():
    m = fa()
    BOUNDS = m._lib.FA_ERR_DEVICE_BOUNDS
    c = case(120, [4, 30, 6], [60, 200, 50], d=128)
    ref = oracle(c, seqs=[0, 2])
    for field, value in (("lens", 201), ("lens", -1), ("prefix", -1)):
        c2 = dict(c, lens=c["lens"].clone())
        kw = {}
        if field == "lens":
            c2["lens"][1] = value
        else:
            kw["prefix_lens"] = torch.tensor([0, value, 0], dtype=torch.int32)
        out, lse, ws = run(c2, check=False, fill=7.0, **kw)
        assert m.fa_check_device_error(ws) == (BOUNDS, 1)
        assert m.fa_check_device_error(ws) == (0, 0)
        assert_close(out, lse, ref)
        assert (out[4:34] == 7).all() and (lse[:, 4:34] == 7).all()
    # a chunk longer than max_seqlen_q; prefix sums that run backwards or past the rows
    out, lse, ws = run(dict(c, max_q=20), check=False, fill=7.0)
    assert m.fa_check_device_error(ws) == (BOUNDS, 1)
    assert_close(out, lse, ref)
    for cu in ([0, 4, 2, 40], [0, 4, 4, 41], [-1, 4, 4, 10]):
        out, lse, ws = run(dict(c, cu=torch.tensor(cu, dtype=torch.int32)), check=False, fill=7.0)
        assert m.fa_check_device_error(ws)[0] == BOUNDS
    # pages outside the cache: recorded, the other sequences right
    for page in (-1, c["kc"].shape[0], 2**31 - 1):
        c2 = dict(c, bt=c["bt"].clone())
        c2["bt"][1, 3] = page
        out, lse, ws = run(c2, check=False)
        rc, info = m.fa_check_device_error(ws)
        assert rc == BOUNDS and info == page % 2**32
        assert_close(out, lse, ref)


def test_workspace_has_to_be_contiguous():
    m = fa()
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in (ws[:256].expand(4096, 256), ws[::2]):
        with pytest.raises(m.FaError) as e:
            m.fa_fwd_chunk(z(1, 1, 1, 64), z(1, 4, 1, 64), z(1, 4, 1, 64), lens, max_seqlen_k=4, workspace=bad)
        assert e.value.status == m._lib.FA_ERR_INVALID_ARG
        with pytest.raises(m.FaError) as e:
            m.fa_kvcache_append(z(1, 1, 1, 64), z(1, 1, 1, 64), z(1, 4, 1, 64), z(1, 4, 1, 64), lens, workspace=bad)
        assert e.value.status == m._lib.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("d,dtype", [(128, BF), (64, H)])
def test_shared_and_repeated_pages(d, dtype):
    # a common beginning of three sequences, and one sequence that holds a page twice
    c = case(160, [5, 40, 1], [90, 90, 1200], d=d, dtype=dtype)
    c["bt"][1, :3] = c["bt"][0, :3]
    c["bt"][2, :3] = c["bt"][0, :3]
    c["bt"][2, 7] = c["bt"][2, 50]
    check(c)


def test_overlapping_rows_past_32_bits():
    # every other sequence claims all 2^20 rows, those between run backwards: 8192 row tiles times 2^19 sequences
    m = fa()
    n, seqs = 2**20, 2**20
    cu = torch.zeros(seqs + 1, dtype=torch.int32)
    cu[1::2] = n
    assert (n // 128) * (seqs // 2) == 2**32
    q = torch.zeros(n, 1, 64, dtype=BF, device="cuda")
    kv = torch.zeros(1, 16, 1, 64, dtype=BF, device="cuda")
    lens = torch.full((seqs,), 16, dtype=torch.int32, device="cuda")
    guard = torch.full((n + 256, 1, 64), 7.0, dtype=BF, device="cuda")
    out, _, ws = m.fa_fwd_chunk(q, kv, kv, lens, out=guard[128:128 + n], cu_seqlens_q=cu.cuda(),
                                block_table=torch.zeros(seqs, 1, dtype=torch.int32, device="cuda"), max_seqlen_q=n,
                                max_seqlen_k=16)
    assert m.fa_check_device_error(ws)[0] == m._lib.FA_ERR_DEVICE_BOUNDS
    assert (guard[:128] == 7).all() and (guard[128 + n:] == 7).all()


def test_small_workspace_and_misaligned_arguments():
    m = fa()
    c = case(125, [4], [60])
    with pytest.raises(m.FaError) as e:
        run(c, workspace=torch.zeros(512, dtype=torch.uint8, device=DEV))
    assert e.value.status == m._lib.FA_ERR_WORKSPACE
    with pytest.raises(m.FaError) as e:
        run(c, alibi_slopes=torch.zeros(3))
    assert e.value.status == m._lib.FA_ERR_INVALID_ARG


def test_wait_that_runs_out_is_reported():
    """The first key tile is never sent (FA_DEBUG_WITHHOLD): the bounded waits
    give up, the status is reported, and the next call on the workspace is right."""
    m = fa()
    c = case(126, [4, 30], [60, 200])
    _, _, ws = run(c, check=False, debug_flags=m.FA_DEBUG_WITHHOLD)
    assert m.fa_check_device_error(ws)[0] == m._lib.FA_ERR_DEVICE_TIMEOUT
    out, lse, _ = run(c, workspace=ws)
    assert_close(out, lse, oracle(c))


def test_far_pages():
    """Pages beyond 2^31 elements of the cache: the append writes them, the attention reads them."""
    m = fa()
    hkv, d, page = 8, 128, 64
    n_pages = 2**31 // (page * hkv * d) + 4
    kc = torch.empty(n_pages, page, hkv, d, dtype=BF, device=DEV)
    vc = torch.empty(n_pages, page, hkv, d, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(130)
    n = 150
    bt = torch.tensor([[n_pages - 1, 1, n_pages - 3]], dtype=torch.int32)
    q, k, v = rnd(g, n, 8, d), rnd(g, n, hkv, d), rnd(g, n, hkv, d)
    cu = torch.tensor([0, n], dtype=torch.int32)
    _, lens, _ = m.fa_kvcache_append(k.to(DEV), v.to(DEV), kc, vc, torch.zeros(1, dtype=torch.int32, device=DEV),
                                     cu_seqlens_q=cu.to(DEV), block_table=bt.to(DEV))
    out, lse, _ = m.fa_fwd_chunk(q.to(DEV), kc, vc, lens, cu_seqlens_q=cu.to(DEV), block_table=bt.to(DEV), max_seqlen_q=n,
                                 max_seqlen_k=n)
    small = torch.zeros(3, page, hkv, d, dtype=BF)
    small_v = torch.zeros(3, page, hkv, d, dtype=BF)
    for p in range(3):
        part = k[p * page:(p + 1) * page]
        small[p, :len(part)], small_v[p, :len(part)] = part, v[p * page:(p + 1) * page]
    c = dict(q=q, kc=small, vc=small_v, lens=torch.tensor([n]), cu=cu, bt=torch.tensor([[0, 1, 2]]), params={})
    assert_close(out, lse, oracle(c))


def test_serving_steps():
    """A prompt in pieces and then tokens, two sequences side by side, with
    rotation: fa_kvcache_append and fa_fwd_chunk step by step against attention
    over the whole rotated sequences."""
    from oracle import attention as A
    from oracle import rotary as R
    m = fa()
    for dtype, d, hq, hkv, page in ((BF, 128, 8, 2, 16), (H, 64, 6, 6, 24)):
        g = torch.Generator().manual_seed(140)
        total = [230, 61]
        q, k, v = ([rnd(g, n, h, d, dtype=dtype) for n in total] for h in (hq, hkv, hkv))
        f, _ = m.fa_rope_inv_freq(d // 2, 10000.0)
        fd = f.to(DEV)
        n_pages = sum(-(-n // page) for n in total) + 1
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        bt = torch.full((2, -(-max(total) // page)), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(total):
            bt[s, :-(-n // page)] = perm[at:at - (-n // page)]
            at += -(-n // page)
        kc = torch.full((n_pages, page, hkv, d), float("nan"), dtype=dtype, device=DEV)
        vc = kc.clone()
        lens = [torch.zeros(2, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)]
        ws = None
        got = [[], []]
        done = [0, 0]
        for step in ([100, 0], [129, 60], [1, 1]):
            rows = [x[s][done[s]:done[s] + step[s]] for x in (q, k, v) for s in (0, 1)]
            qs, ks, vs = torch.cat(rows[:2]).to(DEV), torch.cat(rows[2:4]).to(DEV), torch.cat(rows[4:]).to(DEV)
            cu = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device=DEV)
            done = [a + b for a, b in zip(done, step)]
            if ws is None:
                _, plan = m.fa_fwd_chunk_plan(qs, kc, vc, lens[0], cu_seqlens_q=cu, block_table=bt.to(DEV), max_seqlen_q=200,
                                              max_seqlen_k=max(total))
                ws = m.alloc_workspace(2 * plan["workspace_bytes"], DEV)
            qr, _, _ = m.fa_kvcache_append(ks, vs, kc, vc, lens[0], q=qs, cu_seqlens_q=cu, block_table=bt.to(DEV), inv_freq=fd,
                                           seqlens_out=lens[1], workspace=ws)
            out, _, _ = m.fa_fwd_chunk(qr, kc, vc, lens[1], cu_seqlens_q=cu, block_table=bt.to(DEV), max_seqlen_q=200,
                                       max_seqlen_k=max(total), workspace=ws)
            lens.reverse()
            got[0].append(out[:step[0]])
            got[1].append(out[step[0]:])
        assert m.fa_check_device_error(ws) == (0, 0)
        h = torch.finfo(dtype).eps / 2
        for s, n in enumerate(total):
            pos = np.arange(n)
            qr, kr = R.rope(q[s], pos, f), R.rope(k[s], pos, f)
            ref, _ = A.attention(qr[None], kr[None], v[s].double().numpy()[None], causal=True)
            mass, _ = A.attention(qr[None], kr[None], v[s].double().abs().numpy()[None], causal=True)
            o = torch.cat(got[s]).double().cpu().numpy()
            # q and k are each rounded once more after the rotation: a logit moves by at most
            # 2 h (1 + h) scale sum |q k| <= 2 h * |q| |k| / sqrt(d) (Cauchy-Schwarz), p by that share
            norm = np.linalg.norm(qr, axis=-1).max(axis=1)[:, None] * np.linalg.norm(kr, axis=-1).max() / np.sqrt(d)
            dx = np.exp(2 * 2 * h * (1 + h) * norm)[..., None] - 1  # numerator and denominator
            tol = (h * (mass[0] + np.abs(ref[0])) * (1 + h) + 2e-4 * mass[0] + dx * mass[0]) * (1 + h) + n * 2.0 ** -25 * 6
            assert (np.abs(o - ref[0]) <= tol).all(), np.abs(o - ref[0]).max()


def test_capture_streams_and_changed_lengths():
    """Captured once and replayed with other lengths; two calls at once on two
    streams, each with its own workspace."""
    m = fa()
    c = case(150, [1, 1, 1], [4000, 300, 10], hq=8, hkv=2)
    st = {k: dev(c[k]) for k in ("q", "kc", "vc", "lens", "cu", "bt")}
    out, lse, ws = run(c)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)

    def call(o, l, w, stream=None):
        m.fa_fwd_chunk(st["q"], st["kc"], st["vc"], st["lens"], out=o, lse=l, cu_seqlens_q=st["cu"], block_table=st["bt"],
                       max_seqlen_q=1, max_seqlen_k=4000, workspace=w, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o2, l2, ws)
    for lens in ([4000, 300, 10], [129, 300, 1], [3999, 0, 10]):
        st["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert_close(o2, l2, oracle(dict(c, lens=torch.tensor(lens))), n_keys=4000)
    assert m.fa_check_device_error(ws) == (0, 0)
    st["lens"].copy_(c["lens"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(8):
        s = streams[i % 2]
        with torch.cuda.stream(s):
            w = torch.zeros(ws.numel(), dtype=torch.uint8, device=DEV) if i < 2 else outs[i - 2][2]
            o, l = torch.empty_like(out), torch.empty_like(lse)
            call(o, l, w)
            outs.append((o, l, w))
    torch.cuda.synchronize()
    for o, l, _ in outs:
        assert torch.equal(o, out) and torch.equal(l, lse)
    # a stream's handle that is not the current one; buffers allocated by the call
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l, _ = m.fa_fwd_chunk(st["q"], st["kc"], st["vc"], st["lens"], cu_seqlens_q=st["cu"], block_table=st["bt"], max_seqlen_q=1,
                             max_seqlen_k=4000, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (8, 1), (5, 1), (32, 1), (12, 4)])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, H)])
def test_few_rows(hq, hkv, d, dtype):
    """Units of at most 32 (token, head) rows, whose keys are dealt to the four
    quarters of a tile, beside larger ones: each number of 8-row steps, quarters
    without a key, whole and split, every kind of logit."""
    q_lens, kv = [1, 2, 3, 5, 8, 9, 1, 4, 40], [1, 33, 129, 700, 1000, 2000, 5000, 31, 300]
    slopes = torch.tensor([2.0 ** -(1 + h % 8) for h in range(hq)])
    c = case(200 + hq, q_lens, kv, hq=hq, hkv=hkv, d=d, dtype=dtype, page=16)
    check(c, "plain")
    check(c, "window", window_left=20)
    check(c, "gen", logits=2.0, window_left=600, softcap=20.0)
    pre = torch.tensor([1, 20, 0, 699, 0, 1999, 100, 31, 200], dtype=torch.int32)
    check(c, "prefix", prefix_lens=pre)
    out, lse, _ = run(c, alibi_slopes=slopes)
    assert_close(out, lse, oracle(c, alibi_slopes=slopes), "alibi", logits=2.0, n_keys=5000)


def test_nothing_to_do_and_no_keys():
    m = fa()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    z = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    # no sequence; sequences without rows (with and without room for some); rows without keys, in an empty cache too
    out, lse, ws = m.fa_fwd_chunk(z(3, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), i32(), cu_seqlens_q=i32(0),
                                  block_table=torch.zeros(0, 1, dtype=torch.int32, device=DEV), max_seqlen_q=4, max_seqlen_k=16)
    assert out.shape == (3, 4, 64) and m.fa_check_device_error(ws) == (0, 0)
    for max_q in (0, 4):
        out, _, ws = m.fa_fwd_chunk(z(0, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), i32(5, 0), cu_seqlens_q=i32(0, 0, 0),
                                    block_table=torch.zeros(2, 1, dtype=torch.int32, device=DEV), max_seqlen_q=max_q, max_seqlen_k=16)
        torch.cuda.synchronize()
        assert out.numel() == 0 and m.fa_check_device_error(ws) == (0, 0)
    for pages in (0, 2):
        for max_k in (0, 16) if pages else (0,):
            out, lse, ws = m.fa_fwd_chunk(z(5, 4, 128) + 1, z(pages, 16, 2, 128), z(pages, 16, 2, 128), i32(0, 0),
                                          cu_seqlens_q=i32(0, 2, 5), block_table=torch.full((2, 1), -1, dtype=torch.int32, device=DEV),
                                          max_seqlen_q=3, max_seqlen_k=max_k)
            assert (out == 0).all() and torch.isneginf(lse).all() and m.fa_check_device_error(ws) == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_nan_stays_in_its_row(d):
    """A NaN in one query row makes that row NaN, whole, split or narrow, and no other."""
    for q_lens, kv in (([40, 3], [300, 200]), ([1, 2], [300, 5000]), ([40, 2], [9000, 400])):
        c = case(300, q_lens, kv, d=d, page=16)
        ref = run(c)
        bad = dict(c, q=c["q"].clone())
        bad["q"][1, 2, 5] = float("nan")
        out, lse, _ = run(bad)
        assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[2, 1])
        keep = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
        keep[1, 2] = False
        assert torch.equal(out[keep], ref[0][keep]) and torch.equal(lse.T[keep], ref[1].T[keep])


def few_row_lengths(gp):
    """New tokens per sequence that make 1, 8, 9, 31 and 32 rows of gp heads, where gp divides them."""
    return [n // gp for n in (1, 8, 9, 31, 32) if n % gp == 0 and n >= gp] or [32 // gp]


@pytest.mark.parametrize("hq,hkv,gp", [(2, 2, 1), (4, 2, 2), (3, 1, 3), (8, 2, 4), (5, 1, 5), (8, 1, 8), (9, 1, 9), (16, 1, 16),
                                       (31, 1, 31), (32, 1, 32)])
@pytest.mark.parametrize("d,dtype", [(128, BF), (128, H), (64, BF), (64, H)])
@pytest.mark.parametrize("far", [False, True])
def test_form_for_few_rows(hq, hkv, gp, d, dtype, far):
    """Calls in which no unit has more than 32 (token, head) rows: the keys of a tile are dealt to its four
    quarters.  Up to 1500 keys and (d = 64: the other form; whole and split) up to 5000; every kind of logit."""
    m = fa()
    q_lens = few_row_lengths(gp) * 2
    if max(q_lens) * gp < 32 and 32 // gp not in q_lens:
        q_lens.append(32 // gp)
    lens = [33, 1500, 129, 700, 1, 1000, 31, 97, 128, 260, 600] if not far else [5000, 33, 129, 2500, 1, 300, 4097, 31, 640, 700, 90]
    kv = [max(lens[i % len(lens)], n) for i, n in enumerate(q_lens)]
    c = case(400 + hq, q_lens, kv, hq=hq, hkv=hkv, d=d, dtype=dtype, page=32)
    _, plan = m.fa_fwd_chunk_plan(c["q"], c["kc"], c["vc"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                                  max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"])
    assert plan["rows_per_tile"] == 32 // gp and plan["n_heads_sched"] == hq // gp
    assert c["max_q"] * gp <= 32 and (c["max_k"] > 2048) == far
    slopes = torch.tensor([2.0 ** -(1 + h % 8) for h in range(hq)])
    pre = torch.tensor([(0, 1, 40, 200, 10000)[i % 5] for i in range(len(q_lens))], dtype=torch.int32)
    check(c, "plain")
    check(c, "window", window_left=20)
    check(c, "both windows", causal=False, window_left=200, window_right=3)
    check(c, "prefix", prefix_lens=pre)
    check(c, "soft-cap", logits=2.0, softcap=20.0)
    check(c, "soft-cap and window", logits=2.0, softcap=20.0, window_left=600)
    check(c, "soft-cap and prefix", logits=2.0, softcap=20.0, prefix_lens=pre)
    for kw in ({}, dict(softcap=15.0), dict(prefix_lens=pre), dict(window_left=100)):
        out, lse, _ = run(c, alibi_slopes=slopes, **kw)
        assert_close(out, lse, oracle(c, alibi_slopes=slopes, **kw), f"alibi {list(kw)}", logits=2.0, n_keys=c["max_k"])


def poison(c, s, lo, hi, head, what="kc"):
    """Keys lo .. hi - 1 of sequence s as NaN for one K/V head."""
    page = c["kc"].shape[1]
    for j in range(lo, hi):
        c[what][int(c["bt"][s, j // page]), j % page, head] = float("nan")


@pytest.mark.parametrize("q_lens,kv,narrow", [([40, 3], [700, 200], False), ([2, 3], [700, 200], True),
                                              ([40, 2], [9000, 400], False), ([3, 2], [9000, 400], True)])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, H)])
def test_nan_keys_of_one_tile(q_lens, kv, narrow, d, dtype):
    """Keys that are NaN fill a row's first tile (or a quarter of it) and finite ones
    follow: output and LSE of the rows that keep them are NaN; no other changes."""
    m = fa()
    c = case(310, q_lens, kv, d=d, dtype=dtype)
    _, plan = m.fa_fwd_chunk_plan(c["q"], c["kc"], c["vc"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"],
                                  max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"])
    assert plan["rows_per_tile"] == (16 if narrow else 64) and (plan["n_splits"] > 0) == (kv[0] > 1024)
    ref = run(c)
    for lo, hi in ((0, 128), (0, 32), (96, 128), (0, 256), (128, 256)):
        bad = dict(c, kc=c["kc"].clone())
        poison(bad, 0, lo, hi, 1)
        out, lse, _ = run(bad)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
        hit[:q_lens[0], 2:] = True  # heads 2 and 3 of sequence 0 read K/V head 1, and every row sees the first tiles
        assert torch.isnan(out[hit]).all() and torch.isnan(lse.T[hit]).all(), (lo, hi)
        assert torch.equal(out[~hit], ref[0][~hit]) and torch.equal(lse.T[~hit], ref[1].T[~hit]), (lo, hi)
    # hidden from the first rows by the causal rule, from all rows by a window
    bad = dict(c, kc=c["kc"].clone())
    poison(bad, 0, kv[0] - 1, kv[0], 1)
    out, lse, _ = run(bad)
    hit[:] = False
    hit[q_lens[0] - 1, 2:] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse.T[hit]).all()
    assert torch.equal(out[~hit], ref[0][~hit]) and torch.equal(lse.T[~hit], ref[1].T[~hit])
    bad = dict(c, kc=c["kc"].clone())
    first = kv[0] - q_lens[0] - 300
    poison(bad, 0, first - 20, first, 1)
    ref = run(c, window_left=300)
    out, lse, _ = run(bad, window_left=300)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("d,dtype,q_lens", [(128, BF, [40, 3]), (64, H, [40, 3]), (128, H, [2, 1]), (64, BF, [2, 1])])
def test_soft_caps_far_above_the_logits(d, dtype, q_lens):
    """cap tanh(x / cap) is x itself for a cap far above it, to the rounding of fp32; and caps that
    logits of some hundred reach."""
    c = case(500, q_lens, [700, q_lens[1]], d=d, dtype=dtype)
    for cap in (100.0, 1e3, 1e5, 1e8, 3e38):
        check(c, f"cap {cap}", softcap=cap)
    # logits of a standard deviation of 34; x is off by 34 times as much, and by up to 2e-6 |x| < 1e-3 from tanh
    for cap in (130.0, 500.0):
        check(c, f"cap {cap}", logits=34.0, softcap=cap, scale=3.0)


@pytest.mark.parametrize("q_len,kv,d,dtype", [(1, 1500, 128, BF), (1, 2500, 64, H), (40, 1100, 64, BF), (40, 1100, 128, H)])
def test_many_units_with_a_short_last_round(q_len, kv, d, dtype):
    """More row tiles than the planner keeps in shared memory, whose last round would leave most of the grid idle: its
    units are cut in five to fill it, the others stay whole.  The shortest units of 1100 keys and more have 9 key
    tiles, and a fifth of them saves 7.2, more than a partial and a join cost (5.5); those of 700 have 6, which save
    4.8 and are not cut."""
    n = 152 * 10 + 30
    rng = np.random.default_rng(5)
    lens = rng.integers(kv - 400, kv, n).tolist()
    c = case(600, [q_len] * n, lens, hq=1, hkv=1, d=d, dtype=dtype, page=64)
    out, lse, ws = run(c)
    pieces, slots, splits, tiles = ws[256:272].view(torch.int32).tolist()
    assert tiles == n and pieces == n - splits + slots
    assert (splits, slots) == ((30, 150) if q_len == 1 else (0, 0))
    assert_close(out, lse, oracle(c), n_keys=kv)
