"""The serving and training operators around rotary positions and the paged KV cache, as cases that can be timed and compared.

  rope    q and k rotated by their positions (forward, and the backward pass, which rotates the other way): fa_rope
  append  the new tokens' k rotated and written, with v, into a paged cache, q rotated on the way: fa_kvcache_append
  chunk   attention of a chunk of new tokens per sequence over the paged cache, from one token to long prompts: fa_fwd_chunk

``run`` computes them in plain torch operations, or, where ``own`` is true, through this package's entry points."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
WORKSPACE = 64 << 20


def _rope(name, b, s, hq, hkv, d, rot, interleaved, dtype, inverse, pos_hi):
    """pos_hi 0: every sequence's rows are at positions 0 .. s - 1; otherwise each row has a position of its own below pos_hi."""
    return dict(name=name, op="rope", b=b, s=s, hq=hq, hkv=hkv, d=d, rot=rot, interleaved=interleaved, dtype=dtype, inverse=inverse, pos_hi=pos_hi)


def _append(name, n, q_lo, q_hi, past_lo, past_hi, hq, hkv, d, page, rot, interleaved, dtype, lens):
    return dict(name=name, op="append", n=n, q_lo=q_lo, q_hi=q_hi, past_lo=past_lo, past_hi=past_hi, hq=hq, hkv=hkv, d=d, page=page, rot=rot,
                interleaved=interleaved, dtype=dtype, lens=lens)


def _chunk(name, n, q_lo, q_hi, past_lo, past_hi, hq, hkv, d, page, dtype, lens, window=-1, softcap=0.0, prefix_hi=0, alibi=False):
    return dict(name=name, op="chunk", n=n, q_lo=q_lo, q_hi=q_hi, past_lo=past_lo, past_hi=past_hi, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype,
                lens=lens, window=window, softcap=softcap, prefix_hi=prefix_hi, alibi=alibi)


def listed():
    return [
        # the rotation of one 8192-token training sequence's q and k (the 32 / 8-head layer of the benchmark)
        _rope("rope_train_layer", 1, 8192, 32, 8, 128, 128, False, "bf16", False, 0),
        # its gradient for the 12-head, d = 64 layer (8 x 1024 tokens), rows of packed documents, a part of the head rotated in pairs
        _rope("rope_grad_part", 8, 1024, 12, 12, 64, 32, True, "f16", True, 1024),
        # one new token of one sequence, far out in a long context: latency
        _rope("rope_one_token", 1, 1, 32, 8, 128, 128, False, "bf16", False, 1 << 20),
        # one decoding step of 64 sequences: each appends its token (the benchmark's paged decode batch)
        _append("append_decode_step", 64, 1, 1, 127, 8191, 32, 8, 128, 16, 128, False, "bf16", 1),
        # a scheduler's step of ragged pieces of prompts, odd sizes, a page size that is no power of two
        _append("append_ragged", 7, 1, 301, 0, 1000, 12, 4, 64, 24, 32, True, "f16", 2),
        # four whole prompts enter the cache
        _append("append_prompts", 4, 4096, 4096, 0, 0, 32, 8, 128, 64, 128, False, "bf16", 3),
        # the 700-key cache of the sliding-window example, one token, one head: latency
        _chunk("chunk_one_token", 1, 1, 1, 699, 699, 1, 1, 64, 16, "bf16", 4, window=60),
        # the benchmark's paged decode batch: one token each of 64 sequences, window and soft-cap
        _chunk("chunk_decode_step", 64, 1, 1, 127, 8191, 32, 8, 128, 16, "bf16", 1, window=4096, softcap=30.0),
        # a few speculated tokens to be verified over a long cache: little work per key, ALiBi
        _chunk("chunk_verify_long", 2, 5, 32, 50000, 65000, 32, 8, 128, 64, "bf16", 5, alibi=True),
        # the benchmark's prefill of 512 new tokens over 4096 keys, from a paged cache
        _chunk("chunk_prefill", 4, 512, 512, 3584, 3584, 32, 8, 128, 16, "bf16", 6),
        # prompts' pieces and single tokens in one batch, some prompts with a prefix that is seen both ways
        _chunk("chunk_mixed", 16, 1, 500, 0, 4000, 12, 12, 64, 48, "f16", 7, prefix_hi=900),
        # the last 2048 tokens of a 32768-token prompt
        _chunk("chunk_long_prompt", 1, 2048, 2048, 30720, 30720, 32, 8, 128, 64, "bf16", 8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(("rope", "append", "chunk", "chunk"))
    d = rng.choice((64, 128))
    hq, hkv = rng.choice(((1, 1), (12, 12), (12, 4), (16, 2), (32, 8), (32, 32), (40, 8), (16, 1), (6, 2)))
    dtype = rng.choice(("bf16", "f16"))
    rot = rng.choice((d, d, d // 2, d // 4, 3 * d // 8))
    interleaved = rng.random() < 0.5
    page = rng.choice((8, 16, 24, 32, 48, 64, 128, 256))
    if op == "rope":
        b = _log_int(rng, 1, 16)
        s = min(65536, _log_int(rng, 1, max(1, 8192 * 40 * 128 // (b * (hq + hkv) * d))))
        return _nameless(_rope("", b, s, hq, hkv, d, rot, interleaved, dtype, rng.random() < 0.5, rng.choice((0, 1 << rng.randint(8, 20)))))
    n = _log_int(rng, 1, 64)
    if op == "append":
        q_hi = _log_int(rng, 1, 16384 * 48 * 128 // (n * (hq + 2 * hkv) * d))
        past_hi = min(_log_int(rng, 1, 32768), (1 << 27) // (n * hkv * d))
        return _nameless(_append("", n, rng.randint(1, q_hi), q_hi, rng.randint(0, past_hi), past_hi, hq, hkv, d, page, rot, interleaved, dtype,
                                 rng.randint(0, 10**6)))
    # sequences x heads x rows x keys at most half the largest listed case's, and no more cache than the decoding batch reads
    past_hi = min(_log_int(rng, 1, 65000), 200000000 // (n * hkv * d))
    most = 32 * 2048 * 31744 // (2 * n * hq * (past_hi + 64))
    q_hi = min(_log_int(rng, 1, max(1, min(2048, most))), 20000000 // (n * (hq + hkv) * d))
    return _nameless(_chunk("", n, rng.randint(1, q_hi), q_hi, rng.randint(0, past_hi), past_hi, hq, hkv, d, page, dtype, rng.randint(0, 10**6),
                            window=rng.choice((-1, -1, -1, _log_int(rng, 16, 8192))), softcap=rng.choice((0.0, 0.0, 0.0, 30.0)),
                            prefix_hi=rng.choice((0, 0, 0, _log_int(rng, 2, 2000))), alibi=rng.random() < 0.2))


def _lengths(case):
    """Each sequence's new tokens and cached tokens before them: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["n"])]
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["n"])]
    prefix = [r.randint(0, case.get("prefix_hi", 0)) for _ in range(case["n"])]
    return q, past, prefix


def _inv_freq(rot, device):
    """Frequencies of a base-500000 rotary embedding scaled for long contexts: wavelengths over 8192 tokens are stretched eightfold, those
    under 2048 kept, the ones between blended."""
    f = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    out = []
    for x in f:
        turns = 8192.0 * x / (2.0 * math.pi)
        w = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        out.append((1.0 - w) * x / 8.0 + w * x)
    return torch.tensor(out, dtype=torch.float64, device=device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(t)

    st = {"case": case}
    if case["op"] == "rope":
        b, s = case["b"], case["s"]
        st["q"], st["k"] = randn(b, s, hq, d), randn(b, s, hkv, d)
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        st["positions"] = torch.randint(0, case["pos_hi"], (b, s), generator=g, device=dev, dtype=torch.int32) if case["pos_hi"] else None
        return st
    q_lens, past, prefix = _lengths(case)
    n, page = case["n"], case["page"]
    kv = [a + b for a, b in zip(q_lens, past)]
    pages = [-(-x // page) for x in kv]
    n_pages = sum(pages) + 1
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    owned = torch.arange(max(pages), device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
    table = torch.full((n, max(pages)), -1, dtype=torch.int32, device=dev)
    table[owned] = perm[:sum(pages)]
    cu = [0]
    for x in q_lens:
        cu.append(cu[-1] + x)
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["past"] = torch.tensor(past, dtype=torch.int32, device=dev)
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["table"] = table
    st["max_q"], st["max_k"] = max(q_lens), max(kv)
    st["q"] = randn(cu[-1], hq, d)
    st["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    if case["op"] == "append":
        st["k"], st["v"] = randn(cu[-1], hkv, d), randn(cu[-1], hkv, d)
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        st["k_cache"] = torch.zeros(n_pages, page, hkv, d, dtype=t, device=dev)
        st["v_cache"] = torch.zeros(n_pages, page, hkv, d, dtype=t, device=dev)
    else:
        st["k_cache"], st["v_cache"] = randn(n_pages, page, hkv, d), randn(n_pages, page, hkv, d)
        st["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=dev) if case["prefix_hi"] else None
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device=dev) if case["alibi"] else None
    return st


# ---- plain forms ----

def _cos_sin(positions, inv_freq, inverse=False):
    angle = positions.double()[..., None, None] * inv_freq
    return angle.cos().float(), (-angle.sin() if inverse else angle.sin()).float()


def _rotated(x, cos, sin, interleaved):
    """x [..., heads, d] with its first 2 * cos.shape[-1] columns rotated, in x's type."""
    half = cos.shape[-1]
    f = x.float()
    if interleaved:
        a, b = f[..., 0:2 * half:2], f[..., 1:2 * half:2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:2 * half]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((head, f[..., 2 * half:]), dim=-1).to(x.dtype)


def _rope_plain(st):
    c = st["case"]
    pos = st["positions"] if st["positions"] is not None else torch.arange(c["s"], device=st["q"].device)[None, :]
    cos, sin = _cos_sin(pos, st["inv_freq"], c["inverse"])
    return _rotated(st["q"], cos, sin, c["interleaved"]), _rotated(st["k"], cos, sin, c["interleaved"])


def _rows_of(st):
    """For each packed row its sequence and its place in it."""
    rows = torch.arange(st["q"].shape[0], device=st["q"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu_q"][1:].contiguous(), rows, right=True)
    return seq, rows - st["cu_q"][seq]


def _append_plain(st):
    c = st["case"]
    seq, i = _rows_of(st)
    pos = (st["past"][seq] + i).long()
    cos, sin = _cos_sin(pos, st["inv_freq"])
    page = st["table"][seq, pos // c["page"]].long()
    st["k_cache"][page, pos % c["page"]] = _rotated(st["k"], cos, sin, c["interleaved"])
    st["v_cache"][page, pos % c["page"]] = st["v"]
    return _rotated(st["q"], cos, sin, c["interleaved"]), st["past"] + (st["cu_q"][1:] - st["cu_q"][:-1]), st["k_cache"], st["v_cache"]


def _chunk_plain(st):
    c = st["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    dev = st["q"].device
    q_lens = (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    kv = st["kv_lens"].long()
    j = torch.arange(st["max_k"], device=dev)
    there = j[None, :] < kv[:, None]
    pages = st["table"][:, j // page].long().clamp(min=0)
    k = torch.where(there[:, :, None, None], st["k_cache"][pages, j % page].float(), 0.0)
    v = torch.where(there[:, :, None, None], st["v_cache"][pages, j % page].float(), 0.0)
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
        seen = seen & (j >= at - c["window"])
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
        return {"rope": _rope_plain, "append": _append_plain, "chunk": _chunk_plain}[c["op"]](state)
    import masked_flash_attention_gb300 as fa
    if c["op"] == "rope":
        return fa.fa_rope(state["q"], state["k"], inv_freq=state["inv_freq"], positions=state["positions"], interleaved=c["interleaved"],
                          inverse=c["inverse"])
    if c["op"] == "append":
        q, lens, _ = fa.fa_kvcache_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["past"], q=state["q"],
                                          cu_seqlens_q=state["cu_q"], block_table=state["table"], inv_freq=state["inv_freq"],
                                          interleaved=c["interleaved"], workspace=state["workspace"])
        return q, lens, state["k_cache"], state["v_cache"]
    out, lse, _ = fa.fa_fwd_chunk(state["q"], state["k_cache"], state["v_cache"], state["kv_lens"], cu_seqlens_q=state["cu_q"],
                                  block_table=state["table"], prefix_lens=state["prefix"], window_left=c["window"], softcap=c["softcap"],
                                  alibi_slopes=state["slopes"], causal=True, max_seqlen_q=state["max_q"], max_seqlen_k=state["max_k"],
                                  workspace=state["workspace"])
    return out, lse


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        rows = case["b"] * case["s"]
        return {"bytes": 4 * rows * (hq + hkv) * d + 4 * rows * bool(case["pos_hi"]), "flops": 3 * rows * (hq + hkv) * case["rot"]}
    q_lens, past, prefix = _lengths(case)
    rows = sum(q_lens)
    if case["op"] == "append":
        return {"bytes": 4 * rows * (hq + 2 * hkv) * d + 16 * case["n"], "flops": 3 * rows * (hq + hkv) * case["rot"]}
    pairs = keys = 0
    for q, p, pre in zip(q_lens, past, prefix):
        first = 0 if case["window"] < 0 else max(0, p - case["window"])
        keys += q + p - first
        i = torch.arange(q, dtype=torch.int64) + p
        lo = torch.zeros_like(i) if case["window"] < 0 else (i - case["window"]).clamp(min=0)
        hi = torch.maximum(i, torch.tensor(min(pre, q + p) - 1))
        pairs += int((hi - lo + 1).sum())
    return {"bytes": 4 * rows * hq * d + 4 * rows * hq + 4 * keys * hkv * d, "flops": 4 * d * hq * pairs}


# ---- the definitions in 64 bits ----

def _turned(x, pos, inv_freq, interleaved, sign):
    """Each pair (a, b) of x as the complex number a + ib times e^(i sign pos f)."""
    half = inv_freq.numel()
    angle = sign * pos.double().unsqueeze(-1) * inv_freq
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(-2)
    y = x.double().clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
        y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        pos = st["positions"]
        if pos is None:
            pos = torch.arange(case["s"], device=st["q"].device).expand(case["b"], case["s"])
        sign = -1.0 if case["inverse"] else 1.0
        return tuple(_turned(st[n], pos, st["inv_freq"], case["interleaved"], sign) for n in ("q", "k"))
    q_lens, past, prefix = _lengths(case)
    page = case["page"]
    table = st["table"].tolist()
    starts = st["cu_q"].tolist()
    if case["op"] == "append":
        pos = torch.cat([torch.arange(p, p + q) for q, p in zip(q_lens, past)]).to(st["q"].device)
        q = _turned(st["q"], pos, st["inv_freq"], case["interleaved"], 1.0)
        k = _turned(st["k"], pos, st["inv_freq"], case["interleaved"], 1.0)
        v = st["v"].double()
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        for s, (n_new, p) in enumerate(zip(q_lens, past)):
            at = p
            while at < p + n_new:  # a page at a time
                row, take = at % page, min(page - at % page, p + n_new - at)
                src = starts[s] + at - p
                kc[table[s][at // page], row:row + take] = k[src:src + take]
                vc[table[s][at // page], row:row + take] = v[src:src + take]
                at += take
        return q, None, kc, vc
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((hq, st["q"].shape[0]), float("-inf"), dtype=torch.float64, device=st["q"].device)
    for s, (n_new, p, pre) in enumerate(zip(q_lens, past, prefix)):
        n_keys = n_new + p
        ids = torch.tensor(table[s][:-(-n_keys // page)], device=st["q"].device)
        keys = st["k_cache"][ids].flatten(0, 1)[:n_keys]
        values = st["v_cache"][ids].flatten(0, 1)[:n_keys]
        j = torch.arange(n_keys, device=st["q"].device)
        for r0 in range(0, n_new, 1024):
            r1 = min(n_new, r0 + 1024)
            place = torch.arange(r0, r1, device=st["q"].device)[:, None] + p
            drop = (j > place) & (j >= pre)
            if case["window"] >= 0:
                drop = drop | (j < place - case["window"])
            for h in range(hq):
                kh, vh = keys[:, h * hkv // hq].double(), values[:, h * hkv // hq].double()
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
