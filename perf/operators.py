"""Workloads of the packed (variable-length) attention and of the paged KV cache.

Four operators, each in its plain form (elementary torch operations in fp32, rounded once) and, with
``own`` set, through the library's entry points:

  prefill  attn_fwd_varlen     attention over packed prompts of different lengths, O and LSE
  train    attn_fwd_varlen + attn_bwd_varlen     the same with the gradients of q, k and v
  decode   attn_decode_paged   one new token per sequence over a paged KV cache, O and LSE
  append   attn_cache_append   rows of new K and V written into the pages of their sequences

Sequences are packed token-major ([tokens, heads, d]); sequence s owns the rows cu[s] .. cu[s + 1].
With a causal mask query i of a sequence sees key j iff j <= i + Nkv - Nq. The cache is a pool of pages
[pages, page_size, Hkv, d]; token t of sequence b is row t % page_size of page table[b, t // page_size].
"""
import math
import random

import torch

own = False


# ---- cases ------------------------------------------------------------------------------------------
def _text(lens):
    return " ".join(str(int(n)) for n in lens)


def _ints(text):
    return [int(t) for t in text.split()]


def _spread(rng, n, lo, hi):
    """n lengths between lo and hi, uniform, as text."""
    return _text(rng.randint(lo, hi) for _ in range(n))


def listed():
    r = random.Random(20)
    return [
        # a few short prompts that arrive together (one of them a single token): launch latency
        {"name": "prefill_short", "op": "prefill", "q_lens": "1 17 64", "k_lens": "", "Hq": 8, "Hkv": 2, "d": 64,
         "causal": True},
        # an ordinary serving batch: ragged prompts, GQA 4, odd lengths
        {"name": "prefill_mixed", "op": "prefill", "q_lens": _text([1733, 977, 2048, 311, 129, 1, 640, 1201, 77, 1075]),
         "k_lens": "", "Hq": 32, "Hkv": 8, "d": 128, "causal": True},
        # long documents, one of 8192 tokens: the largest prefill
        {"name": "prefill_long", "op": "prefill", "q_lens": "8192 5003 3001", "k_lens": "", "Hq": 16, "Hkv": 16,
         "d": 128, "causal": True},
        # the last chunk of prompts whose earlier keys are already there (more keys than queries), d = 256
        {"name": "prefill_chunk_d256", "op": "prefill", "q_lens": "512 512 300 37 512", "k_lens": "2048 1537 300 1061 4000",
         "Hq": 8, "Hkv": 4, "d": 256, "causal": True},
        # a small training batch of packed samples
        {"name": "train_small", "op": "train", "q_lens": "200 77 1 513", "k_lens": "", "Hq": 4, "Hkv": 2, "d": 128,
         "causal": True},
        # a training row of about 8192 packed tokens, 16 heads
        {"name": "train_packed", "op": "train", "q_lens": "2048 1500 911 2047 130 64 999 493", "k_lens": "", "Hq": 16,
         "Hkv": 16, "d": 128, "causal": True},
        # one short conversation, the first tokens after its prompt
        {"name": "decode_one", "op": "decode", "k_lens": "129", "page": 16, "cap": 4096, "Hq": 8, "Hkv": 2, "d": 64},
        # a serving batch: lengths far below what the page table has room for
        {"name": "decode_batch", "op": "decode", "k_lens": _spread(r, 64, 1, 4096), "page": 16, "cap": 131072, "Hq": 32,
         "Hkv": 8, "d": 128},
        # long contexts of very different lengths: the largest decode
        {"name": "decode_long", "op": "decode", "k_lens": _spread(r, 8, 1024, 131072), "page": 64, "cap": 131072,
         "Hq": 32, "Hkv": 8, "d": 128},
        # wide heads, eight query heads per kv head
        {"name": "decode_d256", "op": "decode", "k_lens": _spread(r, 16, 1, 8192), "page": 32, "cap": 16384, "Hq": 16,
         "Hkv": 2, "d": 256},
        # one new token of each running sequence goes into the cache
        {"name": "append_tokens", "op": "append", "new": _text([1] * 64), "k_lens": _spread(r, 64, 1, 4096), "page": 16,
         "cap": 131072, "Hkv": 8, "d": 128},
        # a packed batch of prompts goes into the cache
        {"name": "append_prompts", "op": "append", "new": _text([1733, 977, 2048, 311, 129, 1, 640, 1201, 77, 1075]),
         "k_lens": _text([1733, 977, 2048, 311, 129, 1, 640, 1301, 77, 2000]), "page": 16, "cap": 4096, "Hkv": 8,
         "d": 128},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log((hi + 1) / lo))))


def _padded_scores(c, q, k):
    """fp32 bytes of the padded score tensor of the plain form."""
    return 4 * len(q) * c["Hq"] * max(q + [1]) * max(k + [1])


def draw(rng):
    op = rng.choice(["prefill", "train", "decode", "append"])
    c = {"op": op, "Hkv": rng.choice([1, 2, 3, 4, 8]), "d": 128 if op == "train" else rng.choice([32, 64, 128, 128, 256])}
    if op in ("prefill", "train"):
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4] if op == "train" else [1, 2, 3, 4, 8])
        n = _log_int(rng, 1, 32)
        top = _log_int(rng, 1, 2048 if op == "train" else 8192)
        q = [_log_int(rng, 1, top) if rng.random() < 0.95 else 0 for _ in range(n)]
        if sum(q) == 0:
            q[0] = 1
        k = list(q)
        if op == "prefill" and rng.random() < 0.3:  # earlier keys are there already
            k = [a + (_log_int(rng, 1, top) if rng.random() < 0.7 else 0) for a in q]
        c["causal"] = rng.random() < 0.8
        limit, flops, tokens = (1.5e9, 1.8e11, 8192) if op == "train" else (1.2e10, 4.1e11, 16384)
        while (_padded_scores(c, q, k) * max(1, c["d"] / 128) > limit
               or max(sum(q), sum(k)) * c["Hq"] * c["d"] > tokens * 2048
               or work({**c, "q_lens": _text(q), "k_lens": _text(k)})["flops"] > flops):
            q, k = [(a + 1) // 2 for a in q], [(a + 1) // 2 for a in k]
        c.update(q_lens=_text(q), k_lens="" if q == k else _text(k))
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    n = _log_int(rng, 1, 128)
    top = _log_int(rng, 16, 131072 if op == "decode" else 8192)
    k = [_log_int(rng, 1, top) if i == 0 or rng.random() < 0.97 else 0 for i in range(n)]
    while len(k) * max(k + [1]) * c["Hkv"] * c["d"] > 1 << 30 or sum(k) * c["Hkv"] * c["d"] > 1 << 28:
        k = [(a + 1) // 2 for a in k]
    c["k_lens"] = _text(k)
    c["cap"] = -(-max(k + [1]) // c["page"]) * c["page"] * rng.choice([1, 1, 4])
    if op == "decode":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
    elif rng.random() < 0.5:
        c["new"] = _text(min(1, a) for a in k)
    else:
        c["new"] = _text(rng.randint(1 if i == 0 else 0, a) for i, a in enumerate(k))
    return c


# ---- inputs -----------------------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _offsets(lens):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0).to(torch.int32)
    return t.cuda()


def _pool(case, gen, lens):
    """A pool with a few pages to spare, its pages given to the sequences in random order; unused entries
    of the table are -1."""
    page, width = case["page"], case["cap"] // case["page"]
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = _offsets(need).long()
    col = torch.arange(width, device="cuda")
    used = col[None, :] < (first[1:] - first[:-1])[:, None]
    at = (first[:-1, None] + col[None, :]).clamp(max=total - 1)
    table = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
    shape = (total, page, case["Hkv"], case["d"])
    return {"table": table, "k_pages": _normal(gen, *shape), "v_pages": _normal(gen, *shape),
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, d = case["op"], case["d"]
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if op in ("prefill", "train"):
        ql = _ints(case["q_lens"])
        kl = _ints(case["k_lens"]) or ql
        s.update(cu_q=_offsets(ql), cu_k=_offsets(kl), max_q=max(ql), max_k=max(kl),
                 q=_normal(gen, sum(ql), case["Hq"], d), k=_normal(gen, sum(kl), case["Hkv"], d),
                 v=_normal(gen, sum(kl), case["Hkv"], d))
        if op == "train":
            s["dout"] = _normal(gen, sum(ql), case["Hq"], d)
        return s
    lens = _ints(case["k_lens"])
    s.update(_pool(case, gen, lens), max_k=max(lens))
    if op == "decode":
        s["q"] = _normal(gen, len(lens), case["Hq"], d)
    else:
        new = _ints(case["new"])
        s.update(cu=_offsets(new), k_new=_normal(gen, sum(new), case["Hkv"], d),
                 v_new=_normal(gen, sum(new), case["Hkv"], d))
    return s


# ---- plain forms --------------------------------------------------------------------------------------
def _padded(x, cu, longest):
    """Packed rows [T, H, d] as fp32 [S, longest, H, d] (rows past a sequence's end are 0), and which are real."""
    lens = cu[1:] - cu[:-1]
    i = torch.arange(longest, device=x.device)
    real = i[None, :] < lens[:, None]
    at = (cu[:-1, None].long() + i[None, :]).clamp(max=max(x.shape[0] - 1, 0))
    return x[at].float() * real[:, :, None, None], real


def _places(cu, n):
    """Sequence and index within it of each of the n packed rows."""
    t = torch.arange(n, device=cu.device, dtype=torch.int32)
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return s, t.long() - cu[s].long()


def _probabilities(s):
    """P [S, Hkv, G, Lq, Lk] and LSE [S, Hkv, G, Lq], with the padded operands."""
    case = s["case"]
    q, q_real = _padded(s["q"], s["cu_q"], s["max_q"])
    k, k_real = _padded(s["k"], s["cu_k"], s["max_k"])
    S, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1:3]
    q = q.view(S, Lq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)       # [S, Hkv, G, Lq, d]
    k = k.permute(0, 2, 1, 3)[:, :, None]                             # [S, Hkv, 1, Lk, d]
    seen = (q_real[:, :, None] & k_real[:, None, :])
    if case["causal"]:
        shift = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
        i, j = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
        seen &= j[None, None, :] <= i[None, :, None] + shift[:, None, None]
    hidden = ~seen[:, None, None]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log())[..., 0]
    p = p.div_(z.masked_fill(z == 0, 1.0))
    return p, lse, q, k


def _packed_attention(s):
    p, lse, q, k = _probabilities(s)
    v, _ = _padded(s["v"], s["cu_k"], s["max_k"])
    v = v.permute(0, 2, 1, 3)[:, :, None]
    o = torch.matmul(p, v)                                            # [S, Hkv, G, Lq, d]
    return p, lse, q, k, v, o


def _pack(x, cu, n):
    """[S, Hkv, G, L, d] back to packed rows [n, H, d]."""
    b, i = _places(cu, n)
    y = x.permute(0, 3, 1, 2, 4)[b, i]
    return y.reshape(n, -1, x.shape[-1])


def _prefill(s):
    _, lse, _, _, _, o = _packed_attention(s)
    n = s["q"].shape[0]
    o = _pack(o, s["cu_q"], n).to(torch.bfloat16)
    lse = _pack(lse[..., None], s["cu_q"], n)[..., 0].t().contiguous()
    return {"o": o, "lse": lse}


def _train(s):
    p, lse, q, k, v, o = _packed_attention(s)
    n, nk = s["q"].shape[0], s["k"].shape[0]
    do, _ = _padded(s["dout"], s["cu_q"], s["max_q"])
    do = do.view(*do.shape[:2], q.shape[1], q.shape[2], -1).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True) * s["scale"]
    rows = {"o": (o, "cu_q", n), "dq": (dq, "cu_q", n), "dk": (dk, "cu_k", nk), "dv": (dv, "cu_k", nk)}
    return {name: _pack(x, s[cu], m).to(torch.bfloat16) for name, (x, cu, m) in rows.items()}


def _decode(s):
    page = s["k_pages"].shape[1]
    B, Hq, d = s["q"].shape
    Hkv = s["k_pages"].shape[2]
    ids = s["table"][:, :max(1, -(-s["max_k"] // page))].clamp(min=0).long()
    n = ids.shape[1] * page
    k = s["k_pages"][ids].view(B, n, Hkv, d).permute(0, 2, 1, 3).float()
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    hidden = (torch.arange(n, device=q.device)[None, :] >= s["lens"][:, None])[:, None, None]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
    del k
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    v = s["v_pages"][ids].view(B, n, Hkv, d).permute(0, 2, 1, 3).float()
    o = torch.matmul(p, v) / z.masked_fill(z == 0, 1.0)
    return {"o": o.reshape(B, Hq, d).to(torch.bfloat16), "lse": (m + z.log()).reshape(B, Hq)}


def _append(s):
    page = s["k_pages"].shape[1]
    b, i = _places(s["cu"], s["k_new"].shape[0])
    pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[b] + i
    at = s["table"][b, pos // page].long()
    s["k_pages"][at, pos % page] = s["k_new"]
    s["v_pages"][at, pos % page] = s["v_new"]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own(s):
    import exact_io_aware_41_b200 as attn

    op = s["case"]["op"]
    if op == "decode":
        o, lse = attn.attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], scale=s["scale"])
        return {"o": o, "lse": lse}
    if op == "append":
        attn.attn_cache_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                               cu_seqlens=s["cu"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    causal = s["case"]["causal"]
    o, lse = attn.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"], causal=causal)
    if op == "prefill":
        return {"o": o, "lse": lse}
    dq, dk, dv = attn.attn_bwd_varlen(s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu_q"], s["cu_k"],
                                      scale=s["scale"], causal=causal)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    return {"prefill": _prefill, "train": _train, "decode": _decode, "append": _append}[state["case"]["op"]](state)


# ---- the work of a pass, and its outputs in 64 bits -----------------------------------------------------
def work(case):
    """Every operand read once and every result written once (bf16; LSE, offsets and table entries 4 bytes);
    products counted over the visible (query, key) pairs only."""
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] in ("prefill", "train"):
        q = _ints(case["q_lens"])
        k = _ints(case["k_lens"]) or q
        Hq, tq, tk = case["Hq"], sum(q), sum(k)
        seen = 0
        for a, b in zip(q, k):
            off = max(0, b - a) if case["causal"] else 0
            # causal rows see b - a + 1, ..., b keys, the ones below 1 none
            lo = max(0, a - b)
            seen += sum((off + 1, off + a - lo)) * (a - lo) // 2 if case["causal"] else a * b
        size = 2 * (2 * tq * Hq * d + 2 * tk * Hkv * d) + 4 * tq * Hq + 8 * len(q)
        if case["op"] == "prefill":
            return {"bytes": size, "flops": 4 * seen * Hq * d}
        # the training pass reads q, k, v, dout and writes o, dq, dk, dv; 2 + 5 products
        return {"bytes": 2 * (4 * tq * Hq * d + 4 * tk * Hkv * d) + 8 * len(q), "flops": 14 * seen * Hq * d}
    lens = _ints(case["k_lens"])
    pages = sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "decode":
        Hq = case["Hq"]
        return {"bytes": 4 * sum(lens) * Hkv * d + 4 * len(lens) * Hq * d + 4 * len(lens) * Hq + 4 * pages,
                "flops": 4 * sum(lens) * Hq * d}
    new = _ints(case["new"])
    return {"bytes": 8 * sum(new) * Hkv * d + 4 * len(lens) + 4 * sum(-(-n // case["page"]) for n in new), "flops": 0}


def exact(case, seed):
    """The same outputs from the definition, sequence by sequence and head by head in fp64."""
    op = case["op"]
    if op == "append":
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d)
    o = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    if op == "decode":
        lse = torch.full((o.shape[0], Hq), -math.inf, dtype=f64, device="cuda")
        for b, n in enumerate(_ints(case["k_lens"])):
            if n == 0:
                continue
            ids = s["table"][b, :-(-n // case["page"])].long()
            for g in range(Hkv):
                k = s["k_pages"][ids, :, g].reshape(-1, d)[:n].to(f64)
                v = s["v_pages"][ids, :, g].reshape(-1, d)[:n].to(f64)
                x = scale * (s["q"][b, g * G:(g + 1) * G].to(f64) @ k.t())
                lse[b, g * G:(g + 1) * G] = torch.logsumexp(x, 1)
                o[b, g * G:(g + 1) * G] = torch.softmax(x, 1) @ v
        return {"o": o, "lse": lse}
    lse = torch.full((Hq, o.shape[0]), -math.inf, dtype=f64, device="cuda")
    grads = {n: torch.zeros(s[n[1]].shape, dtype=f64, device="cuda") for n in ("dq", "dk", "dv")} if op == "train" else {}
    ql = _ints(case["q_lens"])
    kl = _ints(case["k_lens"]) or ql
    q0 = k0 = 0
    for a, b in zip(ql, kl):
        qr, kr = slice(q0, q0 + a), slice(k0, k0 + b)
        q0, k0 = q0 + a, k0 + b
        if a == 0 or b == 0:
            continue
        unseen = torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1) if case["causal"] else None
        for h in range(Hq):
            g = h // G
            q, k, v = s["q"][qr, h].to(f64), s["k"][kr, g].to(f64), s["v"][kr, g].to(f64)
            x = scale * (q @ k.t())
            if unseen is not None:
                x[unseen] = -math.inf
            z = torch.logsumexp(x, 1)
            lse[h, qr] = z
            p = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            o[qr, h] = p @ v
            if op == "train":
                do = s["dout"][qr, h].to(f64)
                ds = p * (do @ v.t() - (do * o[qr, h]).sum(1, keepdim=True))
                grads["dq"][qr, h] = scale * (ds @ k)
                grads["dk"][kr, g] += scale * (ds.t() @ q)
                grads["dv"][kr, g] += p.t() @ do
    return {"o": o, "lse": lse} if op == "prefill" else {"o": o, **grads}
