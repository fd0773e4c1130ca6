"""Cases and the tolerance of fa_fwd_chunk's tests.

Tolerance.  O = sum p_j v_j / sum p_j with p_j rounded to the input type for the
product (half a step h = eps / 2 relative, so at most h * mass, mass = sum p |v| /
sum p), the result rounded once (h |O|).  fp16's p below 2^-14 are off by up to
2^-25 absolute; the row's largest p is at least 1 (the reference is never above
the maximum), so that adds at most kv_len 2^-25 max|V|, and 2^-25 for the result.
The logits: a dot product of d <= 128 terms in fp32 is off by at most
d 2^-24 sum|q k| scale, for N(0, 1) inputs below 128 * 6e-8 * 82 * 0.09 = 6e-5;
the soft-cap adds 30 * 3e-7 * 1.45 (cap 30); exponent and sums are fp32.  That is
less than 1e-4 relative in p, hence 2e-4 * mass in O, and 1e-4 in LSE, to which
its own fp32 rounding (|LSE| 2^-23) is added.  `logits` scales this for inputs
that are larger than N(0, 1)."""
import numpy as np
import torch

from oracle import chunk as C

BF, H = torch.bfloat16, torch.float16
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def rnd(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(dtype)


def case(seed, q_lens, kv_lens, hq=4, hkv=2, d=128, page=16, dtype=BF, extra=(0, 0), fixed=False, **params):
    """Packed (or, fixed, [B, Sq, ...]) queries over a cache whose unused rows and
    pages hold NaN and whose tables hold -1 past a sequence's keys."""
    g = torch.Generator().manual_seed(seed)
    n = len(q_lens)
    cu = np.concatenate([[0], np.cumsum(q_lens)]) + extra[0]
    q = rnd(g, int(cu[-1]) + extra[1], hq, d, dtype=dtype)
    if page:
        pages = [-(-L // page) for L in kv_lens]
        n_pages = sum(pages) + 2
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        bt = torch.full((n, max(1, max(pages, default=1))), -1, dtype=torch.int32)
        kc = torch.full((n_pages, page, hkv, d), float("nan"), dtype=dtype)
    else:
        bt = None
        kc = torch.full((n, max(kv_lens, default=0) + 3, hkv, d), float("nan"), dtype=dtype)
    vc = kc.clone()
    at = 0
    for s, L in enumerate(kv_lens):
        for c in (kc, vc):
            rows = rnd(g, L, hkv, d, dtype=dtype)
            if page:
                for p in range(pages[s]):
                    bt[s, p] = perm[at + p]
                    part = rows[p * page:(p + 1) * page]
                    c[int(perm[at + p]), :part.shape[0]] = part
            else:
                c[s, :L] = rows
        at += pages[s] if page else 0
    out = dict(q=q, kc=kc, vc=vc, bt=bt, cu=torch.tensor(cu, dtype=torch.int32), lens=torch.tensor(kv_lens, dtype=torch.int32),
               max_q=max(q_lens, default=0), max_k=max(kv_lens, default=0), params=params)
    if fixed:
        out["q"] = q.view(n, q_lens[0], hq, d)
        out["cu"] = None
    return out


def dev(t):
    return t.to(DEV) if isinstance(t, torch.Tensor) else t


def run(c, check=True, fill=None, **kw):
    import masked_flash_attention_gb300 as fa
    p = {k: dev(v) for k, v in {**c["params"], **kw}.items()}
    q = dev(c["q"])
    if fill is not None:
        p["out"] = torch.full_like(q, fill)
        p["lse"] = torch.full((q.shape[1], q.shape[0]) if c["cu"] is not None else (q.shape[0], q.shape[2], q.shape[1]), fill,
                              dtype=torch.float32, device=DEV)
    out, lse, ws = fa.fa_fwd_chunk(q, dev(c["kc"]), dev(c["vc"]), dev(c["lens"]), cu_seqlens_q=dev(c["cu"]),
                                   block_table=dev(c["bt"]), max_seqlen_q=c["max_q"], max_seqlen_k=c["max_k"], **p)
    torch.cuda.synchronize()
    if check:
        assert fa.fa_check_device_error(ws) == (0, 0)
    return out, lse, ws


def oracle(c, seqs=None, **kw):
    p = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in {**c["params"], **kw}.items()}
    return C.attention_chunk(c["q"], c["kc"], c["vc"], c["lens"], cu_seqlens_q=c["cu"], block_table=c["bt"], seqs=seqs, **p)


def assert_close(out, lse, ref, name="", logits=1.0, n_keys=0, v_max=6.0):
    ro, rl, mass = ref
    h = torch.finfo(out.dtype).eps / 2
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    there = ~np.isnan(ro)
    assert np.isnan(rl).any() == (~there).any()
    tol = h * (mass + np.abs(ro)) * (1 + h) + 2e-4 * logits * mass
    if out.dtype == torch.float16:
        tol = tol + n_keys * 2.0 ** -25 * v_max + 2.0 ** -25
    err = np.abs(o - ro)
    bad = there & ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {int(there.sum())} outputs, first {np.argwhere(bad)[0]}, " \
        f"worst {np.nanmax(np.where(bad, err / tol, 0)):.3g} of the tolerance"
    lt = ~np.isnan(rl)
    none = np.isneginf(rl)
    assert np.isneginf(l[none]).all() and np.isfinite(l[lt & ~none]).all(), f"{name}: rows without keys differ"
    le = np.abs(l[lt & ~none] - rl[lt & ~none])
    assert (le <= 1e-4 * logits + np.abs(rl[lt & ~none]) * 2.0 ** -23).all(), f"{name}: LSE off by {le.max()}"


def check(c, name="", logits=1.0, **kw):
    out, lse, _ = run(c, **kw)
    assert_close(out, lse, oracle(c, **kw), name, logits, n_keys=c["max_k"])
    return out, lse
