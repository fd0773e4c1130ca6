"""fa_fwd_chunk on the CPU: pins of its oracle, the plan's geometry, and the
refusals (host-only)."""
import numpy as np
import pytest
import torch

import masked_flash_attention_gb300 as fa
from chunk_util import case, oracle
from masked_flash_attention_gb300 import _lib
from oracle import attention as A
from oracle import chunk as C

BF, H = torch.bfloat16, torch.float16
E, U = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("params", [{}, dict(window_left=5), dict(window_left=3, window_right=0, softcap=5.0), dict(causal=False),
                                    dict(causal=False, window_right=2), dict(alibi_slopes=np.array([0.5, 0.25, 1.0, 2.0]))])
def test_oracle_without_prefix_is_the_paged_oracle(params):
    c = case(1, [3, 0, 7, 1], [9, 4, 7, 20], d=64, page=4)
    cu_k = np.concatenate([[0], np.cumsum(c["lens"].numpy())])
    ref_o, ref_l = A.attention(c["q"], np.nan_to_num(c["kc"].double().numpy()), np.nan_to_num(c["vc"].double().numpy()),
                               cu_seqlens_q=c["cu"], cu_seqlens_k=cu_k, block_table=c["bt"],
                               **{"causal": True, **params})
    o, l, mass = oracle(c, **params)
    assert np.allclose(o, ref_o) and np.allclose(l, ref_l) and (mass >= np.abs(o) - 1e-12).all()


def test_oracle_prefix():
    ok = C.kept(4, 10, prefix=8)
    for i in range(4):
        assert ok[i].tolist() == [j <= i + 6 or j < 8 for j in range(10)]
    # a prefix over all keys is attention without the causal rule
    assert C.kept(5, 9, prefix=9).all() and C.kept(5, 9, prefix=100).all()
    assert (C.kept(5, 9, prefix=3) == C.kept(5, 9)).all()  # the first row sees keys 0 .. 4 anyway
    assert not C.kept(3, 9, prefix=9, window_left=2)[0, 3]  # the window still holds


def test_oracle_more_rows_than_keys():
    ok = C.kept(5, 3)
    assert not ok[:2].any() and ok[2].tolist() == [True, False, False] and ok[4].all()


def T(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def i32(*s):
    return T(*s, dtype=torch.int32)


def plan(q=None, kc=None, vc=None, lens=None, **kw):
    q = T(7, 8, 128) if q is None else q
    kc = T(10, 16, 2, 128) if kc is None else kc
    args = dict(cu_seqlens_q=i32(3), block_table=i32(2, 5), max_seqlen_q=5, max_seqlen_k=80)
    args.update(kw)
    return fa.fa_fwd_chunk_plan(q, kc, kc if vc is None else vc, i32(2) if lens is None else lens, **args)


def test_plan_geometry():
    rc, p = plan()
    assert rc == 0 and p["path"] == _lib.FA_PATH_PREFILL
    # 4 q-heads share a K/V head, 2 head groups; 5 tokens x 4 heads: a query tile of 32 rows
    assert p["rows_per_tile"] == 8 and p["n_heads_sched"] == 2 and p["n_row_tiles"] == 1 and p["n_k_tiles"] == 1
    assert p["n_items"] == 2 * 2 and p["n_kernels"] == 1 and p["n_splits"] == 0  # few, one key tile: nothing to plan or split
    rc, p = plan(block_table=i32(2, 500), max_seqlen_k=8000)
    assert rc == 0 and p["n_k_tiles"] == 63 and p["n_kernels"] == 3 and p["n_splits"] == 4 * 63
    assert p["workspace_bytes"] >= p["n_splits"] * 128 * 129 * 4
    # padded cache, fixed-length queries, nothing to do
    rc, p = plan(T(2, 3, 8, 64), T(2, 40, 2, 64), cu_seqlens_q=None, block_table=None, max_seqlen_k=40)
    assert rc == 0 and p["n_items"] == 4
    rc, p = plan(T(2, 0, 8, 64), T(2, 40, 2, 64), cu_seqlens_q=None, block_table=None, max_seqlen_k=40)
    assert rc == 0 and p["n_items"] == 0 and p["n_kernels"] == 0
    rc, p = plan(T(0, 8, 128), cu_seqlens_q=i32(1), lens=i32(0), block_table=i32(0, 5), max_seqlen_q=0)
    assert rc == 0 and p["n_items"] == 0


@pytest.mark.parametrize("hq,hkv,gp", [(1, 1, 1), (8, 8, 1), (32, 8, 4), (5, 1, 5), (12, 2, 6), (40, 1, 40), (48, 1, 24),
                                       (128, 1, 128), (256, 1, 128), (33, 1, 11), (11, 1, 11), (62, 2, 31)])
def test_plan_heads_per_tile(hq, hkv, gp):
    rc, p = plan(T(7, hq, 64), T(10, 16, hkv, 64), max_seqlen_q=40)
    assert rc == 0 and p["n_heads_sched"] == hq // gp and p["rows_per_tile"] == 128 // gp, (p["n_heads_sched"], p["rows_per_tile"])


def test_plan_refusals():
    bad = [
        plan(T(7, 8, 96), T(10, 16, 2, 96)), plan(T(7, 8, 64)), plan(T(7, 9, 128)), plan(T(7, 8, 128).float()),
        plan(T(7, 8, 128, dtype=H)), plan(vc=T(10, 16, 2, 128, dtype=H)), plan(vc=T(10, 15, 2, 128)),
        plan(T(2, 3, 8, 128)), plan(cu_seqlens_q=None), plan(cu_seqlens_q=i32(4)), plan(cu_seqlens_q=i32(3).long()),
        plan(lens=i32(3)), plan(lens=i32(2).long()), plan(block_table=i32(3, 5)), plan(block_table=i32(2, 5).long()),
        plan(block_table=i32(5, 2).T), plan(block_table=None), plan(max_seqlen_k=81), plan(max_seqlen_k=-1),
        plan(max_seqlen_q=0), plan(prefix_lens=i32(3)), plan(prefix_lens=i32(2), causal=False),
        plan(window_left=-2), plan(window_right=-2), plan(softcap=-1.0), plan(softcap=float("nan")), plan(scale=float("inf")),
        plan(out=T(7, 8, 64)), plan(out=T(7, 8, 128, dtype=H)), plan(out=T(1, 8, 128).expand(7, 8, 128)),
        plan(lse=T(8, 6, dtype=torch.float32)), plan(lse=T(8, 7, dtype=torch.float64)), plan(lse=T(7, 8, dtype=torch.float32)),
        plan(T(7, 8, 256)[..., ::2]), plan(T(7, 8, 132)[..., :128]), plan(kc=T(0, 16, 2, 128)),
        plan(T(2, 3, 8, 64), T(3, 40, 2, 64), cu_seqlens_q=None, block_table=None, max_seqlen_k=40),
        plan(T(2, 3, 8, 64), T(2, 40, 2, 64), cu_seqlens_q=None, block_table=None, max_seqlen_k=41),
    ]
    assert [rc for rc, _ in bad] == [E] * len(bad), [rc for rc, _ in bad]
    uns = [plan(T(1, 8, 128).expand(7, 8, 128), out=T(7, 8, 128)), plan(kc=T(10, 16, 1, 128).expand(10, 16, 2, 128)),
           plan(vc=T(1, 16, 2, 128).expand(10, 16, 2, 128))]
    assert [rc for rc, _ in uns] == [U] * len(uns)


def test_binding_refuses_host_tensors():
    with pytest.raises(fa.FaError):
        fa.fa_fwd_chunk(T(2, 3, 8, 64), T(2, 40, 2, 64), T(2, 40, 2, 64), i32(2), max_seqlen_k=40)


def test_plan_without_planner_only_for_few_short_units():
    kernels = lambda n, q, k: plan(T(n * q, 8, 128), cu_seqlens_q=i32(n + 1), lens=i32(n), block_table=i32(n, 600),  # noqa: E731
                                   max_seqlen_q=q, max_seqlen_k=k)[1]["n_kernels"]
    assert kernels(4, 1, 1024) == 1 and kernels(4, 300, 1024) == 1
    assert kernels(4, 1, 1025) == 3       # more than 8 key tiles: split and joined
    assert kernels(1000, 1, 1024) == 2    # many units: listed by the planner


def test_plan_cuts_only_what_its_sums_hold():
    # one token each of n sequences over 2^18 key tiles (they share their pages): 2^31 tiles and more are not cut
    def splits(n):
        kc = torch.empty(1, 2**20, 1, 64, dtype=BF)
        return plan(T(n, 1, 64), kc, cu_seqlens_q=i32(n + 1), lens=i32(n), block_table=i32(n, 32), max_seqlen_q=1,
                    max_seqlen_k=(2**31 - 1) // 64)

    n_kt = 2**18
    rc, p = splits(2**13 - 1)
    assert rc == 0 and p["n_k_tiles"] == n_kt and p["n_splits"] > 0
    rc, p = splits(2**13 + 1)
    assert rc == 0 and p["n_splits"] == 0 and p["n_kernels"] == 2


def test_plan_refuses_more_row_tiles_than_it_can_count():
    # (strides that overlap, so that the rows need no memory of their own)
    def rows(n):
        return torch.empty(n * 8 + 128 * 8 + 64, dtype=BF).as_strided((n, 128, 64), (8, 8, 1))

    # 128 q-heads share a K/V head: a token per query tile
    many = lambda n: plan(rows(n), T(10, 16, 1, 64), lse=torch.empty(1).as_strided((128, n), (0, 0)),  # noqa: E731
                          cu_seqlens_q=i32(2), lens=i32(1), block_table=i32(1, 5), max_seqlen_q=n)[0]
    assert many(2**22) == 0 and many(2**22 + 1) == E


def test_binding_refuses_none_for_numbers():
    with pytest.raises(TypeError):
        plan(window_left=None)
    with pytest.raises(TypeError):
        plan(softcap=None)
    assert plan(window_left=2**40)[0] == E


def test_max_seqlen_k_is_required():
    """Left out it stood for 0, so that every sequence with keys was recorded as out of bounds on the device."""
    assert plan(max_seqlen_k=None)[0] == E and plan(lens=i32(2), max_seqlen_k=None, cu_seqlens_q=i32(3))[0] == E
    assert fa.fa_fwd_chunk_plan(T(2, 3, 8, 64), T(2, 40, 2, 64), T(2, 40, 2, 64), i32(2))[0] == E
    assert plan(max_seqlen_k=0)[0] == 0  # no sequence has a key
