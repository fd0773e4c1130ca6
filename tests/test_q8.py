"""The KV cache in 8 bits on the CPU: pins of its oracle, the plan's geometry and the
refusals of fa_kvcache_append_q8, fa_kvcache_read_q8 and fa_fwd_chunk_q8."""
import ctypes

import numpy as np
import pytest
import torch

import masked_flash_attention_gb300 as fa
from masked_flash_attention_gb300 import _lib
from oracle import chunk as C
from oracle import q8 as Q
from oracle import rotary as R
from q8_util import cache, chunk_case, codes_of, oracle

BF, H, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
E = _lib.FA_ERR_INVALID_ARG


# ---- the oracle ----

def test_codes_are_the_type_of_torch():
    v = Q.code_values()
    t = torch.arange(256, dtype=torch.uint8).view(E4)
    assert np.array_equal(v, t.double().numpy(), equal_nan=True)
    assert np.array_equal(Q.values(t), v, equal_nan=True)


def test_rounding_to_codes():
    assert Q.to_code([0.0, 448.0, 463.9, 1e9, -1e9]).tolist() == [0.0, 448.0, 448.0, 448.0, -448.0]
    assert Q.to_code([17.0, 19.0, 16.9, 2.0 ** -10, 1.5 * 2.0 ** -9, 2.0 ** -9 * 0.51]).tolist() == [16.0, 20.0, 16.0, 0.0, 2.0 ** -8, 2.0 ** -9]
    assert np.isnan(Q.to_code([np.nan, np.inf, -np.inf])).all()
    x = np.random.default_rng(0).uniform(-450, 450, 20000) * 2.0 ** np.random.default_rng(1).integers(-15, 1, 20000)
    ref = torch.from_numpy(x).clamp(-448, 448).float().to(E4).double().numpy()  # (fp32 first: no ties here)
    assert np.array_equal(Q.to_code(x), ref)


def test_block_exponents():
    assert [Q.exponent(x) for x in (448.0, 448.0001, 1.75, 1.0, 0.0, 1e30, 1e-30)] == [0, 1, -8, -8, -40, 40, -40]


def test_oracle_append_of_a_block_at_once_and_in_pieces():
    """The codes of a block depend on the order only through what its growing scale rounded again."""
    rng = np.random.default_rng(2)
    k = rng.standard_normal((20, 1, 64)) * 2.0 ** rng.integers(-3, 4, (20, 1, 1))
    empty = lambda: (np.full((3, 16, 1, 64), np.nan), np.full((3, 1, 1), np.nan))  # noqa: E731
    bt = np.array([[2, 0]])
    kc, ks = empty()
    once = Q.append(k, k, kc, kc, ks, ks, [0], cu_seqlens_q=[0, 20], block_table=bt)
    c, s, at = kc, ks, 0
    for n in (1, 4, 9, 6):
        r = Q.append(k[at:at + n], k[at:at + n], c, c, s, s, [at], cu_seqlens_q=[0, n], block_table=bt)
        c, s, at = r["k"], r["k_scale"], at + n
    assert np.array_equal(s, once["k_scale"], equal_nan=True)
    big = Q.dequantised(c, s)
    ref = np.full_like(big, np.nan)
    ref[2, :, 0], ref[0, :4, 0] = k[:16, 0], k[16:, 0]
    there = ~np.isnan(ref)
    assert np.array_equal(there, ~np.isnan(big))
    # two roundings: 2^-4 of the value each, or half a subnormal step of the scale
    scale = np.repeat(s, 16, 1)[..., None]
    assert (np.abs(big - ref) <= 2.1 * np.maximum(2.0 ** -4 * np.abs(ref), scale * 2.0 ** -10))[there].all()


def test_oracle_append_without_quantising_is_the_plain_append():
    """What the codes stand for before their rounding is what the append in the model's type writes."""
    rng = np.random.default_rng(3)
    kn, vn, q = (rng.standard_normal((5, h, 64)) for h in (2, 2, 4))
    f = 100.0 ** (-np.arange(16) / 16)
    bt = np.array([[3, 1], [0, 5]])
    kc, s = np.zeros((6, 16, 2, 64)), np.full((6, 1, 2), 2.0 ** -40)
    a = Q.append(kn, vn, kc, kc, s, s, [15, 2], q=q, cu_seqlens_q=[0, 2, 5], block_table=bt, inv_freq=f, mscale=1.5)
    rq, rk, rv, rl = R.kvcache_append(kn, vn, kc, kc, [15, 2], q=q, cu_seqlens_q=[0, 2, 5], block_table=bt, inv_freq=f, mscale=1.5)
    assert np.array_equal(a["q"], rq) and list(a["lens"]) == list(rl)
    for name, ref in (("k", rk), ("v", rv)):
        there = ref != 0
        got = a[name + "_exact"] * np.repeat(a[name + "_scale"], 16, 1)[..., None]
        assert np.allclose(got[there], ref[there], rtol=1e-14)


def test_oracle_masks():
    assert (Q.kept(5, 40, window_left=3, sinks=0) == C.kept(5, 40, window_left=3)).all()
    ok = Q.kept(3, 40, window_left=3, sinks=2)
    assert (ok ^ C.kept(3, 40, window_left=3)).sum(1).tolist() == [2, 2, 2] and ok[:, :2].all()
    assert not Q.kept(2, 1, window_left=0, sinks=4)[0].any()  # the causal rule holds for them too
    assert (Q.kept(4, 30, sinks=5) == C.kept(4, 30)).all()


def test_oracle_attention_is_the_one_over_the_read_back_cache():
    c = chunk_case(4, [3, 0, 7, 1], [9, 4, 40, 20], d=64, page=32, block=16)
    o, l, mass, size = oracle(c, window_left=9, softcap=5.0)
    back = {n: torch.from_numpy(Q.dequantised(c[n], c[n + "_scale"])) for n in "kv"}
    ref = C.attention_chunk(c["q"], back["k"], back["v"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"], window_left=9, softcap=5.0)
    assert np.allclose(o, ref[0]) and np.allclose(l, ref[1]) and np.allclose(mass, ref[2]) and (size > 0).any()


def test_cases_are_codes():
    c = cache(5, [30, 0, 5], page=48, block=16)
    t = codes_of(c["k"])
    assert np.array_equal(Q.values(t), c["k"], equal_nan=True)
    assert np.isnan(c["k_scale"]).any() and not np.isnan(c["k"][int(c["bt"][0, 0]), :30]).any()


# ---- the plan ----

def T(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def i32(*s):
    return T(*s, dtype=torch.int32)


def f32(*s):
    return T(*s, dtype=torch.float32)


def plan(q=None, kc=None, vc=None, ks=None, vs=None, lens=None, **kw):
    q = T(7, 8, 128) if q is None else q
    kc = T(10, 32, 2, 128, dtype=E4) if kc is None else kc
    ks = f32(kc.shape[0], kc.shape[1] // 16, kc.shape[2]) if ks is None else ks
    args = dict(cu_seqlens_q=i32(3), block_table=i32(2, 5), max_seqlen_q=5, max_seqlen_k=160)
    args.update(kw)
    return fa.fa_fwd_chunk_q8_plan(q, kc, kc if vc is None else vc, ks, ks if vs is None else vs, i32(2) if lens is None else lens, **args)


def test_plan_geometry():
    rc, p = plan()
    assert rc == 0 and p["path"] == _lib.FA_PATH_PREFILL and p["n_k_tiles"] == 2 and p["n_splits"] == 0 and p["n_kernels"] == 1
    rc, p = plan(block_table=i32(2, 500), max_seqlen_k=16000)
    assert rc == 0 and p["n_k_tiles"] == 125 and p["n_kernels"] == 3 and p["n_splits"] > 0
    rc, p = plan(T(2, 3, 8, 64), T(2, 64, 2, 64, dtype=E4), cu_seqlens_q=None, block_table=None, max_seqlen_k=64)
    assert rc == 0 and p["n_items"] == 4
    rc, p = plan(T(2, 0, 8, 64), T(2, 64, 2, 64, dtype=E4), cu_seqlens_q=None, block_table=None, max_seqlen_k=64)
    assert rc == 0 and p["n_items"] == 0 and p["n_kernels"] == 0
    for block in (16, 32, 64, 128):
        assert plan(kc=T(10, 128, 2, 128, dtype=E4), ks=f32(10, 128 // block, 2))[0] == 0


@pytest.mark.parametrize("hq", [2, 16, 18, 24, 80])
def test_plan_without_tokens(hq):
    """No tokens, with more heads of a group than a tile of few rows has rows."""
    rc, p = plan(T(2, 0, hq, 64), T(2, 64, 2, 64, dtype=E4), cu_seqlens_q=None, block_table=None, max_seqlen_k=64)
    assert rc == 0 and p["n_items"] == 0 and p["n_kernels"] == 0
    rc, p = plan(T(0, hq, 64), T(10, 32, 2, 64, dtype=E4), max_seqlen_q=0)
    assert rc == 0 and p["n_items"] == 0


def test_plan_of_few_short_units():
    """One launch where a window leaves few tiles and every unit has a CTA; a planner and a join where not."""
    tokens = lambda n, sk, **kw: plan(T(n, 8, 128), cu_seqlens_q=i32(n + 1), block_table=i32(n, 500), lens=i32(n), max_seqlen_q=1,  # noqa: E731
                                      max_seqlen_k=sk, **kw)[1]["n_kernels"]
    assert tokens(2, 16000) == 3 and tokens(2, 16000, window_left=1100) == 1 and tokens(2, 16000, window_left=1700) == 3
    assert tokens(2, 16000, window_left=1100, sink_keys=4) == 1 and tokens(2, 16000, window_left=1100, sink_keys=500) == 3
    assert tokens(2, 16000, window_left=1100, prefix_lens=i32(2)) == 3
    assert tokens(2, 16000, window_left=1100, causal=False, window_right=50) == 1
    assert tokens(2, 16000, window_left=1100, causal=False) == 3
    assert tokens(2, 1400) == 1 and tokens(2, 2000) == 3 and tokens(64, 2000) == 1 and tokens(64, 2100) == 3
    assert tokens(160, 1400) == 3  # more units than CTAs
    assert tokens(2, 16000, window_left=1100, sink_keys=2**31 - 1) == 3


def test_plan_refusals():
    kc = T(10, 32, 2, 128, dtype=E4)
    bad = [
        plan(T(7, 8, 96), T(10, 32, 2, 96, dtype=E4)), plan(T(7, 8, 64)), plan(T(7, 9, 128)), plan(T(7, 8, 128).float()),
        plan(kc=T(10, 32, 2, 128)), plan(vc=T(10, 32, 2, 128)), plan(vc=T(10, 16, 2, 128, dtype=E4), vs=f32(10, 1, 2)),
        plan(kc=kc.view(torch.uint8)), plan(ks=f32(10, 2, 2).half()), plan(ks=f32(10, 2, 1)), plan(ks=f32(9, 2, 2)), plan(ks=f32(10, 2)),
        plan(ks=f32(10, 3, 2)), plan(ks=f32(10, 4, 2)), plan(ks=f32(10, 0, 2)), plan(ks=f32(10, 2, 2), vs=f32(10, 1, 2)),
        plan(kc=T(10, 256, 2, 128, dtype=E4), ks=f32(10, 1, 2)), plan(kc=T(10, 48, 2, 128, dtype=E4), ks=f32(10, 1, 2)),
        plan(kc=T(10, 32, 2, 136, dtype=E4)[..., :128]), plan(kc=T(10, 32, 2, 256, dtype=E4)[..., ::2]), plan(kc=T(0, 32, 2, 128, dtype=E4)),
        plan(T(2, 3, 8, 128)), plan(cu_seqlens_q=None), plan(cu_seqlens_q=i32(4)), plan(lens=i32(3)), plan(lens=i32(2).long()),
        plan(block_table=i32(3, 5)), plan(block_table=i32(2, 5).long()), plan(block_table=i32(5, 2).T), plan(block_table=None),
        plan(max_seqlen_k=161), plan(max_seqlen_k=-1), plan(max_seqlen_k=None), plan(max_seqlen_q=0), plan(prefix_lens=i32(3)),
        plan(prefix_lens=i32(2), causal=False), plan(sink_keys=-1), plan(sink_keys=2**40), plan(window_left=-2), plan(window_right=-2),
        plan(softcap=-1.0), plan(softcap=float("nan")), plan(scale=float("inf")), plan(out=T(7, 8, 64)), plan(out=T(7, 8, 128, dtype=H)),
        plan(out=T(1, 8, 128).expand(7, 8, 128)), plan(lse=f32(8, 6)), plan(lse=T(8, 7, dtype=torch.float64)), plan(T(7, 8, 132)[..., :128]),
        plan(T(2, 3, 8, 64), T(3, 64, 2, 64, dtype=E4), cu_seqlens_q=None, block_table=None, max_seqlen_k=64),
    ]
    assert [rc for rc, _ in bad] == [E] * len(bad), [i for i, (rc, _) in enumerate(bad) if rc != E]
    with pytest.raises(TypeError):
        plan(sink_keys=None)


# ---- refusals of the append and of reading back ----

def _call(fn, tensors, opts):
    args, keep = [], []
    for t in tensors:
        if isinstance(t, (int, float)):
            args.append(t)
            continue
        keep.append(_lib.describe(t))
        args.append(ctypes.byref(keep[-1]) if keep[-1] is not None else None)
    return fn(*args, ctypes.byref(opts))


def word(ws=True):
    opts = _lib.make_opts(stream=0)
    if ws:
        opts.workspace, opts.workspace_bytes = 256, 256
    return opts


def append_rc(kn=None, vn=None, kc=None, vc=None, ks=None, vs=None, lens=None, q=None, q_out=None, cu=None, bt=None, positions=None,
              inv_freq=None, mscale=1.0, qw=None, kw=None, eps=0.0, out=None, ws=True):
    kn = T(2, 3, 2, 64) if kn is None else kn
    vn = kn if vn is None else vn
    kc = T(2, 32, 2, 64, dtype=E4) if kc is None else kc
    vc = T(*kc.shape, dtype=kc.dtype) if vc is None else vc
    ks = f32(kc.shape[0], max(1, kc.shape[1] // 16), kc.shape[2]) if ks is None else ks
    vs = f32(*ks.shape) if vs is None else vs
    lens = i32(2) if lens is None else lens
    return _call(fa.lib.fa_kvcache_append_q8, (q, q_out, kn, vn, kc, vc, ks, vs, cu, lens, bt, positions, inv_freq, mscale, 0, qw, kw, eps,
                                               out), word(ws))


def test_append_refusals():
    pages, bt = T(8, 32, 2, 64, dtype=E4), i32(2, 3)
    q = T(2, 3, 4, 64)
    lens2 = i32(4)
    c = T(2, 32, 2, 64, dtype=E4)
    bad = [
        append_rc(kn=T(2, 3, 2, 96)), append_rc(kn=T(2, 3, 2, 64).float()), append_rc(kn=T(6, 2, 64)),
        append_rc(vn=T(2, 3, 1, 64)), append_rc(vn=T(2, 3, 2, 64).half()),
        append_rc(kc=T(3, 32, 2, 64, dtype=E4)), append_rc(kc=T(2, 32, 4, 64, dtype=E4)), append_rc(kc=T(2, 32, 2, 128, dtype=E4)),
        append_rc(kc=T(2, 32, 2, 64)), append_rc(vc=T(2, 16, 2, 64, dtype=E4), vs=f32(2, 1, 2)), append_rc(vc=c.view(torch.uint8)),
        append_rc(kc=T(2, 1, 2, 64, dtype=E4).expand(2, 32, 2, 64)), append_rc(vc=T(1, 32, 2, 64, dtype=E4).expand(2, 32, 2, 64)),
        append_rc(ks=f32(2, 1, 2).expand(2, 2, 2)), append_rc(vs=f32(1, 2, 2).expand(2, 2, 2)), append_rc(ks=f32(2, 3, 2)),
        append_rc(ks=f32(2, 2, 1)), append_rc(vs=f32(2, 1, 2)), append_rc(ks=f32(2, 4, 2), vs=f32(2, 4, 2)), append_rc(vs=T(2, 2, 2)),
        append_rc(kc=T(2, 24, 2, 64, dtype=E4)), append_rc(kc=T(2, 0, 2, 64, dtype=E4)),
        append_rc(lens=i32(3)), append_rc(lens=T(2, dtype=torch.int64)),
        append_rc(kc=pages, bt=i32(3, 3)), append_rc(kc=pages, bt=i32(2, 0)), append_rc(kc=pages, bt=bt.long()), append_rc(kc=pages, bt=i32(3, 2).T),
        append_rc(q=q), append_rc(q_out=q), append_rc(q=q, q_out=T(2, 3, 2, 64)), append_rc(q=q.half(), q_out=q.half()),
        append_rc(q=T(2, 4, 4, 64), q_out=T(2, 4, 4, 64)), append_rc(positions=i32(2, 2)), append_rc(positions=i32(6)),
        append_rc(inv_freq=T(33, dtype=torch.float64)), append_rc(inv_freq=T(8, dtype=torch.float64), mscale=float("nan")),
        append_rc(eps=-1.0), append_rc(eps=float("nan")), append_rc(eps=float("inf")), append_rc(kw=f32(64)), append_rc(kw=f32(32), eps=1e-6),
        append_rc(qw=f32(64), eps=1e-6), append_rc(q=q, q_out=q, qw=f32(64)), append_rc(q=q, q_out=q, qw=T(64).half(), eps=1e-6),
        append_rc(out=i32(3)), append_rc(lens=lens2[:2], out=lens2[1:3]),
        append_rc(kn=T(6, 2, 64), cu=i32(3, 1)), append_rc(kn=T(6, 2, 64), cu=i32(4)), append_rc(kn=T(2, 3, 2, 64), cu=i32(3)),
    ]
    assert bad == [E] * len(bad), [i for i, rc in enumerate(bad) if rc != E]
    assert append_rc(ws=False) == _lib.FA_ERR_WORKSPACE


def read_rc(kc=None, vc=None, ks=None, vs=None, cu=None, lens=None, bt=None, ko=None, vo=None, ws=True):
    kc = T(2, 32, 2, 64, dtype=E4) if kc is None else kc
    vc = kc if vc is None else vc
    ks = f32(2, 2, 2) if ks is None else ks
    vs = ks if vs is None else vs
    ko = T(2, 5, 2, 64) if ko is None else ko
    vo = T(*ko.shape, dtype=ko.dtype) if vo is None else vo
    return _call(fa.lib.fa_kvcache_read_q8, (kc, vc, ks, vs, cu, lens, bt, ko, vo), word(ws))


def test_read_refusals():
    lens, cu, packed = i32(2), i32(3), T(10, 2, 64)
    bad = [
        read_rc(), read_rc(lens=lens, cu=cu), read_rc(lens=i32(3)), read_rc(lens=lens.long()), read_rc(lens=lens, ko=packed),
        read_rc(cu=cu), read_rc(cu=i32(4), ko=packed), read_rc(cu=i32(3, 1), ko=packed), read_rc(lens=lens, ko=T(2, 5, 1, 64)),
        read_rc(lens=lens, ko=T(2, 5, 2, 128)), read_rc(lens=lens, ko=T(2, 5, 2, 64).float()), read_rc(lens=lens, vo=T(2, 5, 2, 64).half()),
        read_rc(lens=lens, vo=T(2, 6, 2, 64)), read_rc(lens=lens, ko=T(1, 5, 2, 64).expand(2, 5, 2, 64)), read_rc(lens=lens, ks=f32(2, 3, 2)),
        read_rc(lens=lens, vs=f32(2, 1, 2)), read_rc(lens=lens, kc=T(3, 32, 2, 64, dtype=E4), ks=f32(3, 2, 2)), read_rc(lens=lens, kc=T(2, 32, 2, 64)),
        read_rc(lens=lens, bt=i32(3, 3)), read_rc(lens=lens, bt=i32(2, 3).long()), read_rc(lens=lens, bt=i32(2, 0)),
    ]
    assert bad == [E] * len(bad), [i for i, rc in enumerate(bad) if rc != E]
    assert read_rc(lens=lens, ws=False) == _lib.FA_ERR_WORKSPACE


def test_bindings_refuse_host_tensors():
    c, s, n = T(1, 16, 2, 64, dtype=E4), f32(1, 1, 2), i32(1)
    for call in (lambda: fa.fa_kvcache_append_q8(T(1, 2, 2, 64), T(1, 2, 2, 64), c, c, s, s, n), lambda: fa.fa_kvcache_read_q8(c, c, s, s, n, max_seqlen_k=4),
                 lambda: fa.fa_fwd_chunk_q8(T(1, 2, 4, 64), c, c, s, s, n, max_seqlen_k=4), lambda: fa.fa_kvcache_read_q8(c, c, s, s, n, dtype=torch.float32)):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.status == E
