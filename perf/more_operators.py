"""The operators around a KV cache held in 8 bits, and the norms of queries and keys, as cases that can be timed and compared.

  norm    q and k normalised for each head, weighted and rotated by their positions in one pass: fa_qk_norm_rope
  grad    its gradients, those of the two weights among them: fa_qk_norm_rope_bwd
  append  the new tokens' k (normalised, rotated) and v quantised into a paged 8-bit cache, q beside them: fa_kvcache_append_q8
  read    sequences' keys and values read back from that cache: fa_kvcache_read_q8
  chunk   attention of a chunk of new tokens per sequence over that cache, with windows and first keys that stay visible: fa_fwd_chunk_q8

The 8-bit cache: e4m3 values, and for each block of ``block`` tokens of a page and each head one scale, a power of two.

``run`` computes them in plain torch operations, or, where ``own`` is true, through this package's entry points."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
LOWEST, HIGHEST = -40, 40  # exponents of the scales
EPS = 1e-6
WORKSPACE = 64 << 20


def _norm(name, b, s, hq, hkv, d, rot, interleaved, dtype, wtype, pos_hi, grad=False):
    """pos_hi 0: every sequence's rows are at positions 0 .. s - 1; otherwise each row has a position of its own below pos_hi."""
    return dict(name=name, op="grad" if grad else "norm", b=b, s=s, hq=hq, hkv=hkv, d=d, rot=rot, interleaved=interleaved, dtype=dtype, wtype=wtype,
                pos_hi=pos_hi)


def _append(name, n, q_lo, q_hi, past_lo, past_hi, hq, hkv, d, page, block, rot, interleaved, dtype, norm, lens):
    return dict(name=name, op="append", n=n, q_lo=q_lo, q_hi=q_hi, past_lo=past_lo, past_hi=past_hi, hq=hq, hkv=hkv, d=d, page=page, block=block,
                rot=rot, interleaved=interleaved, dtype=dtype, norm=norm, lens=lens)


def _read(name, n, past_lo, past_hi, hkv, d, page, block, dtype, lens):
    return dict(name=name, op="read", n=n, q_lo=0, q_hi=0, past_lo=past_lo, past_hi=past_hi, hq=hkv, hkv=hkv, d=d, page=page, block=block, dtype=dtype,
                lens=lens)


def _chunk(name, n, q_lo, q_hi, past_lo, past_hi, hq, hkv, d, page, block, dtype, lens, window=-1, sinks=0, softcap=0.0, prefix_hi=0, alibi=False):
    return dict(name=name, op="chunk", n=n, q_lo=q_lo, q_hi=q_hi, past_lo=past_lo, past_hi=past_hi, hq=hq, hkv=hkv, d=d, page=page, block=block,
                dtype=dtype, lens=lens, window=window, sinks=sinks, softcap=softcap, prefix_hi=prefix_hi, alibi=alibi)


def listed():
    return [
        # q and k of one 8192-token training sequence (the 32 / 8-head layer of the benchmark) between their projections and the attention
        _norm("norm_train_layer", 1, 8192, 32, 8, 128, 128, False, "bf16", "bf16", 0),
        # one new token of one sequence, far out in a long context: latency
        _norm("norm_one_token", 1, 1, 32, 8, 128, 128, False, "bf16", "f32", 1 << 20),
        # the gradients of that training layer
        _norm("grad_train_layer", 1, 8192, 32, 8, 128, 128, False, "bf16", "bf16", 0, grad=True),
        # the gradients of the 12-head, d = 64 layer, odd lengths of packed documents, a part of the head rotated in pairs
        _norm("grad_part", 7, 613, 12, 12, 64, 32, True, "f16", "f32", 2048, grad=True),
        # one decoding step of 64 sequences (the benchmark's paged decode batch): each token enters a block that others have begun
        _append("append_decode_step", 64, 1, 1, 127, 8191, 32, 8, 128, 16, 16, 128, False, "bf16", False, 1),
        # four whole prompts enter the cache, normalised on the way
        _append("append_prompts", 4, 4096, 4096, 0, 0, 32, 8, 128, 64, 32, 128, False, "bf16", True, 3),
        # the decoding batch's cache read back, as for a move to another cache
        _read("read_batch", 64, 128, 8192, 8, 128, 16, 16, "bf16", 1),
        # a few short ragged sequences, pages of 96
        _read("read_ragged", 5, 1, 700, 4, 64, 96, 32, "f16", 2),
        # one token over a long stream of which a window and the first four keys stay visible: latency
        _chunk("chunk_one_token", 1, 1, 1, 20000, 20000, 8, 2, 64, 16, 16, "bf16", 4, window=1023, sinks=4),
        # the benchmark's paged decode batch: one token each of 64 sequences, window and soft-cap
        _chunk("chunk_decode_step", 64, 1, 1, 127, 8191, 32, 8, 128, 16, 16, "bf16", 1, window=4096, softcap=30.0),
        # prompts' pieces and single tokens in one batch, some prompts with a prefix that is seen both ways
        _chunk("chunk_mixed", 16, 1, 500, 0, 4000, 12, 12, 64, 48, 16, "f16", 7, prefix_hi=900),
        # the benchmark's prefill of 512 new tokens over 4096 keys
        _chunk("chunk_prefill", 4, 512, 512, 3584, 3584, 32, 8, 128, 64, 64, "bf16", 6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(("norm", "grad", "append", "read", "chunk", "chunk"))
    d = rng.choice((64, 128))
    hq, hkv = rng.choice(((1, 1), (12, 12), (12, 4), (16, 2), (32, 8), (32, 32), (40, 8), (16, 1), (6, 2)))
    dtype = rng.choice(("bf16", "f16"))
    rot = rng.choice((d, d, d // 2, d // 4, 3 * d // 8))
    interleaved = rng.random() < 0.5
    block = rng.choice((16, 16, 32, 64, 128))
    page = block * rng.choice((1, 1, 2, 3))
    if op in ("norm", "grad"):
        b = _log_int(rng, 1, 16)
        s = min(65536, _log_int(rng, 1, max(1, 8192 * 40 * 128 // (b * (hq + hkv) * d))))
        return _nameless(_norm("", b, s, hq, hkv, d, rot, interleaved, dtype, rng.choice((dtype, "f32")), rng.choice((0, 1 << rng.randint(8, 20))),
                               grad=op == "grad"))
    n = _log_int(rng, 1, 64)
    if op == "append":
        q_hi = _log_int(rng, 1, 16384 * 48 * 128 // (n * (hq + 2 * hkv) * d))
        past_hi = min(_log_int(rng, 1, 32768), (1 << 27) // (n * hkv * d))
        return _nameless(_append("", n, rng.randint(1, q_hi), q_hi, rng.randint(0, past_hi), past_hi, hq, hkv, d, page, block, rot, interleaved, dtype,
                                 rng.random() < 0.5, rng.randint(0, 10**6)))
    if op == "read":
        past_hi = min(_log_int(rng, 1, 65000), 250000000 // (n * hkv * d))
        return _nameless(_read("", n, rng.randint(1, past_hi), past_hi, hkv, d, page, block, dtype, rng.randint(0, 10**6)))
    # sequences x heads x rows x keys at most those of the prefill, and no more cache than the decoding batch reads
    past_hi = min(_log_int(rng, 1, 65000), 250000000 // (n * hkv * d))
    most = 4 * 32 * 512 * 4096 // (n * hq * (past_hi + 64))
    q_hi = min(_log_int(rng, 1, max(1, min(2048, most))), 20000000 // (n * (hq + hkv) * d))
    window = rng.choice((-1, -1, _log_int(rng, 16, 8192)))
    return _nameless(_chunk("", n, rng.randint(1, q_hi), q_hi, rng.randint(0, past_hi), past_hi, hq, hkv, d, page, block, dtype, rng.randint(0, 10**6),
                            window=window, sinks=rng.choice((0, 0, rng.randint(1, 200))), softcap=rng.choice((0.0, 0.0, 0.0, 30.0)),
                            prefix_hi=rng.choice((0, 0, 0, _log_int(rng, 2, 2000))), alibi=rng.random() < 0.2))


def _lengths(case):
    """Each sequence's new tokens, cached tokens before them and prefix: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["n"])]
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["n"])]
    prefix = [r.randint(0, case.get("prefix_hi", 0)) for _ in range(case["n"])]
    return q, past, prefix


def _inv_freq(rot, device):
    """Frequencies of a base-500000 rotary embedding."""
    return torch.tensor([500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=device)


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, of the scales' range (the lowest for 0)."""
    m, e = torch.frexp(top)
    e = e.int() - 9 + (m > 0.875).int()
    return torch.where(top > 0, e, LOWEST).clamp(LOWEST, HIGHEST)


def _power(e):
    """2^e, by the bits of a float."""
    return ((e.int() + 127) << 23).view(torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape, spread=1.0):
        """Normal values; each head's channels have sizes of their own, as those of projections do."""
        x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
        return (x * (spread ** torch.randn(*shape[-2:], generator=g, device=dev, dtype=torch.float32))).to(t)

    def weight(wtype):
        return (1.0 + 0.2 * torch.randn(d, generator=g, device=dev, dtype=torch.float32)).to(DTYPES[wtype])

    st = {"case": case}
    if case["op"] in ("norm", "grad"):
        b, s = case["b"], case["s"]
        st["q"], st["k"] = randn(b, s, hq, d, spread=1.5), randn(b, s, hkv, d, spread=1.5)
        st["q_weight"], st["k_weight"] = weight(case["wtype"]), weight(case["wtype"])
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        st["positions"] = torch.randint(0, case["pos_hi"], (b, s), generator=g, device=dev, dtype=torch.int32) if case["pos_hi"] else None
        if case["op"] == "grad":
            st["dq_out"], st["dk_out"] = randn(b, s, hq, d), randn(b, s, hkv, d)
            st["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
        return st
    q_lens, past, prefix = _lengths(case)
    n, page, block = case["n"], case["page"], case["block"]
    kv = [a + b for a, b in zip(q_lens, past)]
    pages = [-(-x // page) for x in kv]
    n_pages = sum(pages) + 1
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    owned = torch.arange(max(pages), device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
    table = torch.full((n, max(pages)), -1, dtype=torch.int32, device=dev)
    table[owned] = perm[:sum(pages)]
    cu, cu_k = [0], [0]
    for x, y in zip(q_lens, kv):
        cu.append(cu[-1] + x)
        cu_k.append(cu_k[-1] + y)
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device=dev)
    st["past"] = torch.tensor(past, dtype=torch.int32, device=dev)
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["table"] = table
    st["max_q"], st["max_k"], st["total_k"] = max(q_lens), max(kv), cu_k[-1]
    st["n_blocks"] = sum((p + q - 1) // block - p // block + 1 for q, p in zip(q_lens, past) if q)
    st["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    for name in ("k", "v"):  # what the cache holds already: normal values whose size differs from page to page and head to head
        x = torch.randn(n_pages, page // block, block, hkv, d, generator=g, device=dev, dtype=torch.float32)
        x *= 1.5 ** torch.randn(n_pages, page // block, 1, hkv, 1, generator=g, device=dev, dtype=torch.float32)
        x *= 1.5 ** torch.randn(hkv, d, generator=g, device=dev, dtype=torch.float32)
        e = _exponent(x.abs().amax(dim=(2, 4)))
        x *= _power(-e)[:, :, None, :, None]
        st[name + "_cache"] = x.to(E4M3).view(n_pages, page, hkv, d)
        st[name + "_scale"] = _power(e)
        del x
    if case["op"] == "append":
        st["q"], st["k"], st["v"] = randn(cu[-1], hq, d, spread=1.5), randn(cu[-1], hkv, d, spread=1.5), randn(cu[-1], hkv, d, spread=1.5)
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        st["q_weight"], st["k_weight"] = (weight(case["dtype"]), weight(case["dtype"])) if case["norm"] else (None, None)
    elif case["op"] == "chunk":
        st["q"] = randn(cu[-1], hq, d)
        st["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=dev) if case["prefix_hi"] else None
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device=dev) if case["alibi"] else None
    return st


# ---- plain forms ----

def _cos_sin(positions, inv_freq):
    angle = positions.double()[..., None, None] * inv_freq
    return angle.cos().float(), angle.sin().float()


def _rotated(f, cos, sin, interleaved):
    """f [..., heads, d] in 32 bits with its first 2 * cos.shape[-1] columns rotated."""
    half = cos.shape[-1]
    if interleaved:
        a, b = f[..., 0:2 * half:2], f[..., 1:2 * half:2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:2 * half]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((head, f[..., 2 * half:]), dim=-1)


def _inverse_rms(f):
    return torch.rsqrt((f * f).mean(dim=-1, keepdim=True) + EPS)


def _positions(st):
    return st["positions"] if st["positions"] is not None else torch.arange(st["case"]["s"], device=st["q"].device)[None, :]


def _normed_rotated(x, w, cos, sin, interleaved):
    f = x.float()
    return _rotated(f * _inverse_rms(f) * w.float(), cos, sin, interleaved)


def _norm_plain(st):
    c = st["case"]
    cos, sin = _cos_sin(_positions(st), st["inv_freq"])
    return (_normed_rotated(st["q"], st["q_weight"], cos, sin, c["interleaved"]).to(st["q"].dtype),
            _normed_rotated(st["k"], st["k_weight"], cos, sin, c["interleaved"]).to(st["k"].dtype))


def _grad_of(x, dy, w, cos, sin, interleaved):
    f = x.float()
    r = _inverse_rms(f)
    g = _rotated(dy.float(), cos, -sin, interleaved)  # of the weighted row
    unit = f * r
    dw = (g * unit).flatten(0, 2).sum(dim=0, dtype=torch.float64).float()
    gw = g * w.float()
    return (r * (gw - unit * (gw * unit).mean(dim=-1, keepdim=True))).to(x.dtype), dw


def _grad_plain(st):
    c = st["case"]
    cos, sin = _cos_sin(_positions(st), st["inv_freq"])
    dq, dwq = _grad_of(st["q"], st["dq_out"], st["q_weight"], cos, sin, c["interleaved"])
    dk, dwk = _grad_of(st["k"], st["dk_out"], st["k_weight"], cos, sin, c["interleaved"])
    return dq, dk, dwq, dwk


def _rows_of(st):
    """For each packed row its sequence and its place in it."""
    rows = torch.arange(st["q"].shape[0], device=st["q"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu_q"][1:].contiguous(), rows, right=True)
    return seq, rows - st["cu_q"][seq]


def _touched(st):
    """The blocks that the new rows enter: for each its sequence and its tokens' places in it."""
    block = st["case"]["block"]
    past, kv = st["past"].long(), st["kv_lens"].long()
    first = past // block
    counts = torch.where(kv > past, (kv - 1) // block - first + 1, 0)
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device=past.device), counts, output_size=st["n_blocks"])
    nth = torch.arange(st["n_blocks"], device=past.device) - (counts.cumsum(0) - counts)[seq]
    return seq, ((first[seq] + nth) * block)[:, None] + torch.arange(block, device=past.device)


def _enter(st, seq, at, x, cache, scale):
    """Rows x (32 bits) into their places of the cache; the rows before them in their blocks take the block's new scale."""
    c = st["case"]
    past, kv = st["past"].long()[seq][:, None], st["kv_lens"].long()[seq][:, None]
    new, old = (at >= past) & (at < kv), at < past
    page = st["table"][seq, at[:, 0] // c["page"]].long()
    row, part = at % c["page"], at[:, 0] % c["page"] // c["block"]
    src = (st["cu_q"].long()[seq][:, None] + at - past).clamp(0, x.shape[0] - 1)
    y = torch.where(new[:, :, None, None], x[src], 0.0)
    y = torch.where(y.isfinite(), y, float("nan"))
    e = _exponent(y.nan_to_num(0.0).abs().amax(dim=(1, 3)))
    s = _power(e)
    before = scale[page, part]
    s = torch.where(old.any(dim=1)[:, None], torch.maximum(before, s), s)
    held = cache.view(torch.uint8)[page[:, None], row].view(E4M3).float()
    y = torch.where(new[:, :, None, None], y / s[:, None, :, None], held * (before / s)[:, None, :, None])
    code = y.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    there = new | old
    cache.view(torch.uint8)[page[:, None].expand_as(at)[there], row[there]] = code[there]
    scale[page, part] = s


def _append_plain(st):
    c = st["case"]
    seq, i = _rows_of(st)
    cos, sin = _cos_sin((st["past"][seq] + i).long(), st["inv_freq"])
    if c["norm"]:
        q = _normed_rotated(st["q"], st["q_weight"], cos, sin, c["interleaved"])
        k = _normed_rotated(st["k"], st["k_weight"], cos, sin, c["interleaved"])
    else:
        q, k = _rotated(st["q"].float(), cos, sin, c["interleaved"]), _rotated(st["k"].float(), cos, sin, c["interleaved"])
    seq, at = _touched(st)
    _enter(st, seq, at, k, st["k_cache"], st["k_scale"])
    _enter(st, seq, at, st["v"].float(), st["v_cache"], st["v_scale"])
    return q.to(st["q"].dtype), st["past"] + (st["cu_q"][1:] - st["cu_q"][:-1]), st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]


def _values(st, name, pages, rows):
    """The values, in 32 bits, that the cache holds at these rows of these pages."""
    code = st[name + "_cache"].view(torch.uint8)[pages, rows].view(E4M3).float()
    return code * st[name + "_scale"][pages, rows // st["case"]["block"]][..., None]


def _read_plain(st):
    c = st["case"]
    rows = torch.arange(st["total_k"], device=st["table"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu_k"][1:].contiguous(), rows, right=True)
    at = (rows - st["cu_k"][seq]).long()
    pages = st["table"][seq, at // c["page"]].long()
    t = DTYPES[c["dtype"]]
    return _values(st, "k", pages, at % c["page"]).to(t), _values(st, "v", pages, at % c["page"]).to(t)


def _chunk_plain(st):
    c = st["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    dev = st["q"].device
    q_lens = (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    kv = st["kv_lens"].long()
    j = torch.arange(st["max_k"], device=dev)
    there = j[None, :] < kv[:, None]
    pages = st["table"][:, j // page].long().clamp(min=0)
    k = torch.where(there[:, :, None, None], _values(st, "k", pages, (j % page).expand_as(pages)), 0.0)
    v = torch.where(there[:, :, None, None], _values(st, "v", pages, (j % page).expand_as(pages)), 0.0)
    i = torch.arange(st["max_q"], device=dev)
    rows = (st["cu_q"][:-1].long()[:, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (hkv, hq // hkv))
    x = torch.einsum("nihgd,njhd->nhgij", q, k)
    x *= 1.0 / math.sqrt(d)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    at = i[None, :, None] + (kv - q_lens)[:, None, None]
    if st["slopes"] is not None:
        x -= st["slopes"].view(1, hkv, hq // hkv, 1, 1) * (at - j).abs().float()[:, None, None]
    seen = j <= at
    if st["prefix"] is not None:
        seen = seen | (j < st["prefix"].long()[:, None, None])
    if c["window"] >= 0:
        seen = seen & ((j >= at - c["window"]) | (j < c["sinks"]))
    x.masked_fill_(~(seen & there[:, None, :])[:, None, None], float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    x -= top
    x.exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.einsum("nhgij,njhd->nihgd", x, v)
    some = (total > 0)
    o = torch.where(some.permute(0, 3, 1, 2, 4), o / total.permute(0, 3, 1, 2, 4), 0.0).flatten(2, 3)
    lse = torch.where(some, top + total.log(), float("-inf"))[..., 0].flatten(1, 2)
    seq, at_row = _rows_of(st)
    return o[seq, at_row].to(st["q"].dtype), lse[seq, :, at_row].T.contiguous()


def run(state):
    c = state["case"]
    if not own:
        return {"norm": _norm_plain, "grad": _grad_plain, "append": _append_plain, "read": _read_plain, "chunk": _chunk_plain}[c["op"]](state)
    import masked_flash_attention_gb300 as fa
    if c["op"] == "norm":
        return fa.fa_qk_norm_rope(state["q"], state["k"], q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS, inv_freq=state["inv_freq"],
                                  positions=state["positions"], interleaved=c["interleaved"])
    if c["op"] == "grad":
        return fa.fa_qk_norm_rope_bwd(state["dq_out"], state["dk_out"], state["q"], state["k"], q_weight=state["q_weight"], k_weight=state["k_weight"],
                                      eps=EPS, inv_freq=state["inv_freq"], positions=state["positions"], interleaved=c["interleaved"],
                                      workspace=state["workspace"])[:4]
    cache = state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"]
    if c["op"] == "append":
        q, lens, _ = fa.fa_kvcache_append_q8(state["k"], state["v"], *cache, state["past"], q=state["q"], cu_seqlens_q=state["cu_q"],
                                             block_table=state["table"], inv_freq=state["inv_freq"], interleaved=c["interleaved"],
                                             q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS if c["norm"] else None,
                                             workspace=state["workspace"])
        return q, lens, *cache
    if c["op"] == "read":
        return fa.fa_kvcache_read_q8(*cache, cu_seqlens_k=state["cu_k"], total_k=state["total_k"], block_table=state["table"], dtype=DTYPES[c["dtype"]],
                                     workspace=state["workspace"])[:2]
    out, lse, _ = fa.fa_fwd_chunk_q8(state["q"], *cache, state["kv_lens"], cu_seqlens_q=state["cu_q"], block_table=state["table"],
                                     prefix_lens=state["prefix"], window_left=c["window"], sink_keys=c["sinks"], softcap=c["softcap"],
                                     alibi_slopes=state["slopes"], causal=True, max_seqlen_q=state["max_q"], max_seqlen_k=state["max_k"],
                                     workspace=state["workspace"])
    return out, lse


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("norm", "grad"):
        rows, wide = case["b"] * case["s"], 4 if case["wtype"] == "f32" else 2
        elements = rows * (hq + hkv) * d
        rest = 4 * rows * bool(case["pos_hi"]) + 4 * case["rot"] + 2 * d * (wide + (4 if case["op"] == "grad" else 0))
        return {"bytes": (6 if case["op"] == "grad" else 4) * elements + rest, "flops": (16 if case["op"] == "grad" else 7) * elements}
    q_lens, past, prefix = _lengths(case)
    rows = sum(q_lens)
    if case["op"] == "append":
        scales = 8 * hkv * sum((p + q - 1) // case["block"] - p // case["block"] + 1 for q, p in zip(q_lens, past) if q)
        return {"bytes": rows * (4 * hq + 6 * hkv) * d + scales + 16 * case["n"], "flops": rows * (hq + hkv) * d * (7 if case["norm"] else 3) + 4 * rows * hkv * d}
    if case["op"] == "read":
        return {"bytes": sum(past) * hkv * 6 * d + 8 * hkv * sum(-(-p // case["block"]) for p in past), "flops": 2 * sum(past) * hkv * d}
    pairs = keys = 0
    for q, p, pre in zip(q_lens, past, prefix):
        sinks = case["sinks"] if case["window"] >= 0 else 0
        first = 0 if case["window"] < 0 else max(0, p - case["window"])
        keys += q + p - first + min(first, sinks)
        i = torch.arange(q, dtype=torch.int64) + p
        lo = torch.zeros_like(i) if case["window"] < 0 else (i - case["window"]).clamp(min=0)
        hi = torch.maximum(i, torch.tensor(min(pre, q + p) - 1))
        pairs += int((hi - lo + 1 + lo.clamp(max=sinks)).sum())
    return {"bytes": 4 * rows * hq * d + 4 * rows * hq + 2 * keys * hkv * d + 8 * hkv * keys // case["block"], "flops": 4 * d * hq * pairs}


# ---- the definitions in 64 bits ----

def _turned(y, pos, inv_freq, interleaved, sign=1.0):
    """Each pair (a, b) of y (64 bits) as the complex number a + ib times e^(i sign pos f)."""
    half = inv_freq.numel()
    angle = sign * pos.double().unsqueeze(-1) * inv_freq
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(-2)
    y = y.clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
        y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def _exact_norm(x, w):
    x = x.double()
    return x / torch.sqrt(x.pow(2).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def _exact_grad(x, dy, w, pos, inv_freq, interleaved):
    """y = x n^(-1/2) w with n = mean(x^2) + eps: dx = n^(-1/2) gw - n^(-3/2) x <x, gw> / d."""
    x, w = x.double(), w.double()
    g = _turned(dy.double(), pos, inv_freq, interleaved, -1.0)
    n = x.pow(2).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS
    dw = torch.einsum("bshd,bshd->d", g, x / n.sqrt())
    gw = g * w
    return gw / n.sqrt() - x * (x * gw).sum(dim=-1, keepdim=True) / (x.shape[-1] * n.pow(1.5)), dw


def _exact_entered(case, st, x, name, starts, table, q_lens, past):
    """The cache's codes before their rounding to e4m3 and its scales, block by block of each sequence."""
    page, block = case["page"], case["block"]
    codes, scale = st[name + "_cache"].double(), st[name + "_scale"].double()
    powers = torch.tensor([2.0 ** e for e in range(LOWEST, HIGHEST + 1)], dtype=torch.float64, device=x.device)
    for s, (n_new, p) in enumerate(zip(q_lens, past)):
        rows = x[starts[s]:starts[s] + n_new]
        at = p
        while at < p + n_new:
            begin = at - at % block
            end = min(begin + block, p + n_new)
            pg, r0, b = table[s][begin // page], begin % page, begin % page // block
            mine = rows[at - p:end - p]
            top = mine.abs().amax(dim=(0, 2))
            new = torch.where(powers[:, None] * 448.0 >= top, powers[:, None], math.inf).amin(dim=0)
            new = new.clamp(max=2.0 ** HIGHEST)
            if at > begin:
                new = torch.maximum(new, scale[pg, b])
                codes[pg, r0:r0 + at - begin] *= (scale[pg, b] / new)[None, :, None]
            codes[pg, r0 + at - begin:r0 + end - begin] = mine / new[None, :, None]
            scale[pg, b] = new
            at = end
    return codes, scale


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["inv_freq"].device if "inv_freq" in st else st["table"].device
    if case["op"] in ("norm", "grad"):
        pos = st["positions"]
        if pos is None:
            pos = torch.arange(case["s"], device=dev).expand(case["b"], case["s"])
        if case["op"] == "norm":
            return tuple(_turned(_exact_norm(st[n], st[n + "_weight"]), pos, st["inv_freq"], case["interleaved"]) for n in ("q", "k"))
        (dq, dwq), (dk, dwk) = (_exact_grad(st[n], st["d" + n + "_out"], st[n + "_weight"], pos, st["inv_freq"], case["interleaved"]) for n in ("q", "k"))
        return dq, dk, dwq, dwk
    q_lens, past, prefix = _lengths(case)
    page, block = case["page"], case["block"]
    table = st["table"].tolist()
    starts = st["cu_q"].tolist()
    if case["op"] == "append":
        if st["n_blocks"] > 4000:  # (the loop over the blocks is slow)
            return None
        pos = torch.cat([torch.arange(p, p + q) for q, p in zip(q_lens, past)]).to(dev)
        q, k = (_exact_norm(st[n], st[n + "_weight"]) if case["norm"] else st[n].double() for n in ("q", "k"))
        q, k = (_turned(x, pos, st["inv_freq"], case["interleaved"]) for x in (q, k))
        kc, ks = _exact_entered(case, st, k, "k", starts, table, q_lens, past)
        vc, vs = _exact_entered(case, st, st["v"].double(), "v", starts, table, q_lens, past)
        return q, None, kc, vc, ks, vs

    def held(name, s, n_keys):
        ids = torch.tensor(table[s][:-(-n_keys // page)], device=dev)
        x = st[name + "_cache"].view(torch.uint8)[ids].view(E4M3).double()
        return (x * st[name + "_scale"][ids].double().repeat_interleave(block, dim=1)[..., None]).flatten(0, 1)[:n_keys]

    if case["op"] == "read":
        return tuple(torch.cat([held(n, s, p) for s, p in enumerate(past)]) for n in ("k", "v"))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full((hq, st["q"].shape[0]), float("-inf"), dtype=torch.float64, device=dev)
    for s, (n_new, p, pre) in enumerate(zip(q_lens, past, prefix)):
        n_keys = n_new + p
        keys, values = held("k", s, n_keys), held("v", s, n_keys)
        j = torch.arange(n_keys, device=dev)
        for r0 in range(0, n_new, 1024):
            r1 = min(n_new, r0 + 1024)
            place = torch.arange(r0, r1, device=dev)[:, None] + p
            drop = (j > place) & (j >= pre)
            if case["window"] >= 0:
                drop = drop | ((j < place - case["window"]) & (j >= case["sinks"]))
            for h in range(hq):
                kh, vh = keys[:, h * hkv // hq], values[:, h * hkv // hq]
                score = (st["q"][starts[s] + r0:starts[s] + r1, h].double() @ kh.T) / math.sqrt(d)
                if case["softcap"]:
                    score = torch.tanh(score / case["softcap"]) * case["softcap"]
                if st["slopes"] is not None:
                    score = score - float(st["slopes"][h]) * (place - j).abs()
                score = score.masked_fill(drop, float("-inf"))
                total = torch.logsumexp(score, dim=1)
                out[starts[s] + r0:starts[s] + r1, h] = torch.exp(score - total[:, None]) @ vh
                lse[h, starts[s] + r0:starts[s] + r1] = total
    return out, lse
