"""Cases, checks and tolerances of the operators on an 8-bit cache.

Append.  V, and K without norm and rotation, are quantised from values that fp32
holds exactly, times a power of two: codes and scales have to be the oracle's,
bit for bit, and so have the codes that a growing scale rounds again.  A normalised
or rotated K carries its fp32 error (rope_util and norm_error below) into the
rounding: a code may be off the exact quotient by half a step of e4m3 (2^-4
relative, at least 2^-10) and that error over the scale, and a scale may differ
where the block's largest element lies within that error of a border.

Attention.  The products' inputs are exact in fp16 but for Q's elements under
2^-32 of their row's largest (counted with the logits).  A logit is a sum of d
products in fp32, off by at most d 2^-24 size, size = scale sum |q k|, and three
factors and a sum round by 2^-24 each, as does the exponent: delta = (d + 8) 2^-24
size + 1e-6 (|x| stays below size), with a soft-cap 3e-7 * cap * 1.45 more (the
rounding near 1 of its quotient form; above 128 it follows a power series good to
1e-7 of the logit).  ALiBi adds 2^-23 of the distance term.  O = sum w c / sum
w 2^-b: the fp16 weights are off by 2^-11 relative, or, under 2^-14, by 2^-25
against a top weight of 2^7 or more and codes of at most 448 = twice the block's
largest element: n_keys 2^-31 v_max in all.  So |O - ref| <= h |O| + (2^-11 +
2 delta + 2e-6) mass + n_keys 2^-31 v_max, with h half a step of the output's
type (fp16: its smallest subnormal's half, 2^-25, too).  The fp32 sums of n
positive terms add up to 64 in one accumulator, then the lanes, warps and pieces:
2e-6 covers 32 roundings.  LSE: delta + 2e-6 + |LSE| 2^-23."""
import numpy as np
import torch

from oracle import q8 as Q

BF, H = torch.bfloat16, torch.float16
E4 = torch.float8_e4m3fn
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=BF, spread=0.0):
    x = torch.randn(*shape, generator=g, dtype=torch.float32)
    if spread:
        x = x * 2.0 ** (spread * torch.randn(*shape[:-1], 1, generator=g, dtype=torch.float32))
    return x.to(dtype)


def dev(t):
    return t.to(DEV) if isinstance(t, torch.Tensor) else t


def codes_of(values):
    """fp64 code values as a float8 tensor (each is one of e4m3's)."""
    return torch.from_numpy(np.ascontiguousarray(values)).to(torch.float32).to(E4)


def quantised(x, block):
    """x [pages, page, H, d] fp64 as (code values, scales): NaN rows stay NaN and count for nothing."""
    p, rows, h, d = x.shape
    y = x.reshape(p, rows // block, block, h, d)
    top = np.nan_to_num(np.abs(y)).max(axis=(2, 4))
    s = np.vectorize(lambda t: 2.0 ** Q.exponent(t))(top)
    return Q.to_code(y / s[:, :, None, :, None]).reshape(x.shape), s


def cache(seed, kv_lens, hkv=2, d=128, page=16, block=16, spread=1.0, spare=2):
    """A paged (or, page None, padded) cache of random contents: code 0x7f (NaN) in every row that no sequence has,
    scales of NaN where no sequence has a row, and tables that hold -1 past a sequence's pages."""
    g = gen(seed)
    n = len(kv_lens)
    if page:
        pages = [-(-L // page) for L in kv_lens]
        perm = torch.randperm(sum(pages) + spare, generator=g).to(torch.int32)
        bt = torch.full((n, max(1, max(pages, default=1))), -1, dtype=torch.int32)
        shape = (sum(pages) + spare, page, hkv, d)
    else:
        cap = -(-(max(kv_lens, default=0) + 1) // block) * block
        bt, pages, shape = None, [1] * n, (n, cap, hkv, d)
    full = {}
    for name in "kv":
        x = np.full(shape, np.nan)
        at = 0
        for s, L in enumerate(kv_lens):
            rows = rnd(g, L, hkv, d, dtype=torch.float32, spread=spread).double().numpy()
            if page:
                for p in range(pages[s]):
                    bt[s, p] = perm[at + p]
                    part = rows[p * page:(p + 1) * page]
                    x[int(perm[at + p]), :part.shape[0]] = part
                at += pages[s]
            else:
                x[s, :L] = rows
        code, sc = quantised(x, block)
        used = ~np.isnan(x).all(-1).reshape(shape[0], shape[1] // block, block, hkv).all(2)
        full[name], full[name + "_scale"] = code, np.where(used, sc, np.nan)
    return dict(bt=bt, **full)


def on_device(c):
    out = {n: codes_of(c[n]).to(DEV) for n in "kv"}
    out.update({n + "_scale": torch.from_numpy(c[n + "_scale"]).float().to(DEV) for n in "kv"})
    return out["k"], out["v"], out["k_scale"], out["v_scale"]


def chunk_case(seed, q_lens, kv_lens, hq=4, hkv=2, d=128, page=16, block=16, dtype=BF, extra=(0, 0), fixed=False, **params):
    c = cache(seed, kv_lens, hkv, d, page, block)
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + extra[0]
    q = rnd(gen(seed + 1), int(cu[-1]) + extra[1], hq, d, dtype=dtype)
    c.update(q=q, cu=torch.tensor(cu, dtype=torch.int32), lens=torch.tensor(kv_lens, dtype=torch.int32),
             max_q=max(q_lens, default=0), max_k=max(kv_lens, default=0), params=params)
    if fixed:
        c["q"], c["cu"] = q.view(len(q_lens), q_lens[0], hq, d), None
    return c


def run(c, check=True, on=None, fill=None, **kw):
    import masked_flash_attention_gb300 as fa
    p = {k: dev(v) for k, v in {**c["params"], **kw}.items()}
    q = dev(c["q"])
    if fill is not None:
        p["out"] = torch.full_like(q, fill)
        p["lse"] = torch.full((q.shape[1], q.shape[0]) if c["cu"] is not None else (q.shape[0], q.shape[2], q.shape[1]), fill,
                              dtype=torch.float32, device=DEV)
    out, lse, ws = fa.fa_fwd_chunk_q8(q, *(on_device(c) if on is None else on), dev(c["lens"]), cu_seqlens_q=dev(c["cu"]),
                                      block_table=dev(c["bt"]), max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"], **p)
    torch.cuda.synchronize()
    if check:
        assert fa.fa_check_device_error(ws) == (0, 0)
    return out, lse, ws


def oracle(c, **kw):
    p = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in {**c["params"], **kw}.items()}
    return Q.attention_chunk(c["q"], Q.dequantised(c["k"], c["k_scale"]), Q.dequantised(c["v"], c["v_scale"]), c["lens"],
                             cu_seqlens_q=c["cu"], block_table=c["bt"], **p)


def assert_close(c, out, lse, ref, name="", **kw):
    p = {**c["params"], **kw}
    ro, rl, mass, size = ref
    d, h = out.shape[-1], torch.finfo(out.dtype).eps / 2
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    cap = p.get("softcap", 0.0)
    delta = (d + 8) * 2.0 ** -24 * size + 1e-6 + (3e-7 * 1.45 * cap if cap <= 128 else 0.0)
    if p.get("alibi_slopes") is not None:
        delta = delta + 2.0 ** -23 * c["max_k"] * float(p["alibi_slopes"].max())
    at = np.moveaxis(delta, 0, 1) if c["cu"] is not None else np.moveaxis(delta, 1, 2)  # rows, heads
    v_max = np.nanmax(np.abs(Q.dequantised(c["v"], c["v_scale"])), initial=0.0)
    nan = np.isnan(ro) & ~np.isnan(mass)
    there = ~np.isnan(ro)
    tol = h * np.abs(ro) + (2.0 ** -11 + 2 * at[..., None] + 2e-6) * (1 + h) * mass + c["max_k"] * 2.0 ** -31 * v_max
    if out.dtype == H:
        tol = tol + 2.0 ** -25
    assert np.isnan(o[nan]).all(), f"{name}: NaN lost"
    bad = there & ~(np.abs(o - ro) <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {int(there.sum())} outputs, first {np.argwhere(bad)[0]}, " \
        f"worst {np.nanmax(np.where(bad, np.abs(o - ro) / tol, 0)):.3g} of the tolerance"
    none, lt = np.isneginf(rl), ~np.isnan(rl)
    assert np.isneginf(l[none]).all() and np.isfinite(l[lt & ~none]).all(), f"{name}: rows without keys differ"
    some = lt & ~none
    le, lim = np.abs(l[some] - rl[some]), (delta + 2e-6 + np.abs(np.where(some, rl, 0.0)) * 2.0 ** -23)[some]
    assert (le <= lim).all(), f"{name}: LSE off by {(le / lim).max():.3g} of the tolerance"


def check(c, name="", **kw):
    out, lse, _ = run(c, **kw)
    assert_close(c, out, lse, oracle(c, **kw), name, **kw)
    return out, lse
