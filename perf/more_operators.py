"""Cases of the operators of prompts, of the cache held in 4 bits, and of scoring.

A case's "op" says which:
  "prompt"    causal attention over whole packed prompts, alone or behind keys of earlier turns;
  "cache"     new tokens rotated, quantised into the 4-bit paged cache, and the
              sequences' keys and values read back as packed 16-bit rows;
  "attn4"     attention of a few new tokens per sequence over the 4-bit paged cache;
  "logprobs"  log probabilities of given tokens, entropy and the top alternatives.
`run` computes the plain form in 32 bits with elementary torch operations, or,
where `own` is true, calls this package's kernels.  `exact` is the same from the
definitions in 64 bits, one sequence at a time.

Sizes: 20 query heads over 5 key heads of 128 columns are the framework's
layer (q 2560, k and v 640 rows); the other head layouts are generic.

The cache's format: a vector of D columns is D/2 bytes, columns 2i and 2i + 1 in the
low and high half of byte i, and per 64 columns a pair (s, z) of fp16: a column of
code c stands for s c + z.  Of a group's values, clamped to +-65504, z is the
least rounded to fp16 and s = (greatest - least) / 15 rounded to fp32, then fp16;
c = (x - z) (1/s) rounded to the nearest whole number within 0..15, ties to even, each
operation rounded to fp32.  A key's rotation a cos - b sin rounds each product and the
difference to fp32, so that both sides have the same codes.  (Keys are not normed here: a
norm's sum may be added up in any order, and a last bit of it moves some values
across the border of two codes.)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 64


def listed():
    p = {"op": "prompt", "hq": 20, "hkv": 5, "d": 128, "dtype": "bf16", "past_min": 0, "past_max": 0}
    c = {"op": "cache", "hq": 20, "hkv": 5, "d": 128, "rot": 128, "page": 64, "dtype": "bf16", "src": "fp32",
         "pairs": False, "norm": False, "packed": False, "ragged": False}
    a = {"op": "attn4", "hq": 20, "hkv": 5, "d": 128, "page": 64, "dtype": "bf16", "ragged": False}
    g = {"op": "logprobs"}
    return [
        # one question of a few hundred tokens: latency
        dict(p, name="prompt-one", b=1, n_min=700, n_max=700),
        # prompts that came in together, of one token to a few thousand, half heads
        dict(p, name="prompt-ragged", b=40, n_min=1, n_max=2101, hq=24, hkv=8, d=64, dtype="fp16"),
        # the next turns of four conversations, behind the keys of the turns before
        dict(p, name="prompt-turns", b=4, n_min=500, n_max=1003, past_min=2500, past_max=9000),
        # the largest: one long document
        dict(p, name="prompt-long", b=1, n_min=16384, n_max=16384),
        # drafted tokens of a batch between two products of a decode step
        dict(c, name="cache-drafts", b=61, t=6, own_min=9, own_max=300, hq=24, hkv=8, d=64, rot=48, page=16,
             dtype="fp16", pairs=True, norm=True, ragged=True),
        # prompts straight from the products, packed, and read back for the prompt attention
        dict(c, name="cache-prompts", b=6, t=4500, own_min=2500, own_max=4500, packed=True),
        # one short conversation, one token: latency
        dict(a, name="attn4-one-short", b=1, t=1, prefix=0, own_min=700, own_max=700),
        # drafted tokens of a batch behind one system prompt, ragged, odd prefix, 16-token pages
        dict(a, name="attn4-drafts", b=24, t=5, prefix=8005, own_min=6, own_max=1500, hq=24, hkv=8, d=64, page=16,
             dtype="fp16", ragged=True),
        # two long documents, one token each: few rows over a long axis
        dict(a, name="attn4-two-long", b=2, t=1, prefix=0, own_min=90000, own_max=131001),
        # the largest batch: 64 conversations of 6000 to 16000 tokens
        dict(a, name="attn4-full-batch", b=64, t=1, prefix=0, own_min=6000, own_max=16000),
        # the drafts of one step scored: latency
        dict(g, name="logprobs-few", rows=6, vocab=32000, top=5, dtype="fp32", masked=0.0),
        # a prompt scored over a large vocabulary, some of it not allowed
        dict(g, name="logprobs-prompt", rows=2048, vocab=131072, top=20, dtype="bf16", masked=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "cache", "attn4", "attn4", "logprobs"])
    dtype = rng.choice(["bf16", "fp16"])
    hq, hkv, d = rng.choice([(20, 5, 128), (32, 8, 128), (16, 8, 64), (24, 8, 64), (8, 1, 128), (7, 7, 64)])
    if op == "prompt":
        b = _log(rng, 1, 48)
        # b hq n (n + past) within the largest listed case
        room = 20 * 16384 * 16384 // (2 * b * hq)
        n = min(_log(rng, 2, 12000), int(math.isqrt(room)))
        past = rng.choice([0, 0, _log(rng, 1, 20000)])
        past = max(0, min(past, room // n - n))
        return {"op": op, "b": b, "n_min": rng.choice([1, n // 2 + 1, n]), "n_max": n, "past_min": past // 2,
                "past_max": past, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype}
    page = rng.choice([16, 32, 64, 128])
    if op == "cache":
        b = _log(rng, 1, 96)
        t = min(_log(rng, 1, 4096), max(1, 12000 // b))
        lo = t + rng.choice([0, rng.randrange(0, 200)])
        return {"op": op, "b": b, "t": t, "own_min": lo, "own_max": lo + rng.randrange(0, 60), "hq": hq, "hkv": hkv,
                "d": d, "rot": rng.choice([d, d, d // 2, d - 16]), "page": page, "dtype": dtype,
                "src": rng.choice(["fp32", dtype]), "pairs": rng.random() < 0.3, "norm": rng.random() < 0.4,
                "packed": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    if op == "attn4":
        b = _log(rng, 1, 128)
        t = rng.choice([1, 1, 1, 2, 3, 5, 8])
        # rows times keys within the largest listed case
        room = 2400000 // (max(hkv, hq // 4) * b * t)
        hi = max(t, min(_log(rng, 16, 120000), room + t))
        prefix = rng.choice([0, 0, min(_log(rng, 64, 16384), room // 2 + 1)])
        return {"op": op, "b": b, "t": t, "prefix": prefix, "own_min": max(t, hi // rng.choice([1, 2, 4])),
                "own_max": hi, "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype,
                "ragged": rng.random() < 0.4}
    vocab = _log(rng, 2000, 131072)
    return {"op": op, "rows": min(_log(rng, 1, 2048), 134217728 // vocab), "vocab": vocab,
            "top": rng.choice([0, 1, 5, 20]), "dtype": rng.choice(["fp32", "bf16", "fp16"]),
            "masked": rng.choice([0.0, 0.0, 0.3])}


def _spread(lo, hi, b):
    """b lengths from lo to hi, the last of them hi, in a scattered order."""
    return [lo + (hi - lo) * ((37 * i + 11) % b + 1) // b for i in range(b)] if b > 1 else [hi]


def _lens(case):
    """Own lengths of the sequences, from the case alone (work() counts them)."""
    return _spread(case["own_min"], case["own_max"], case["b"])


def _new(case):
    """Valid new tokens of the sequences: all t (packed: what the own length has room for), or ragged 1..t."""
    b, t = case["b"], case["t"]
    new = [1 + ((i + 1) * 2654435761 >> 9) % t for i in range(b)] if case["ragged"] else [t] * b
    return [min(n, m) for n, m in zip(new, _lens(case))] if case.get("packed") else new


def _queries(case):
    """(queries, keys) of each prompt: log-spread from n_min to n_max, behind past_min to past_max."""
    b, lo, hi = case["b"], case["n_min"], case["n_max"]
    nq = [max(1, int(round(lo * (hi / lo) ** (((37 * i + 11) % b + 1) / b)))) for i in range(b)] if b > 1 else [hi]
    past = _spread(case["past_min"], case["past_max"], b)
    return nq, [n + p for n, p in zip(nq, past)]


def _starts(n, dev):
    return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(device=dev, dtype=torch.int32)


def _paged(case, g, dev):
    """Page ids of the prefix and the sequences, scattered over the cache."""
    lens, page = _lens(case), case["page"]
    need = [-(-n // page) for n in lens]
    npre = -(-case.get("prefix", 0) // page)
    pages = sum(need) + npre + 3
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((case["b"], max(need)), dtype=torch.int32, device=dev)
    col = torch.arange(max(need), device=dev)
    first = torch.tensor([npre + sum(need[:i]) for i in range(len(need))], device=dev)
    n = torch.tensor(need, device=dev)
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.where(col[None, :] < n[:, None], ids[at], table)
    return pages, ids[:npre].contiguous(), table.contiguous(), ids[-1].long()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    rand = lambda *n: torch.randn(*n, generator=g, device=dev)  # noqa: E731
    if own:
        import bit_plane_select_gb300 as trit
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if case["op"] == "logprobs":
        n, v, k, dt = case["rows"], case["vocab"], case["top"], DTYPES[case["dtype"]]
        s["logits"] = torch.empty((n, v), dtype=dt, device=dev)
        step = max(1, (1 << 26) // v)
        for i in range(0, n, step):
            s["logits"][i:i + step] = (2.5 * rand(min(step, n - i), v)).to(dt)
        if case["masked"]:
            s["logits"][:, torch.rand(v, generator=g, device=dev) < case["masked"]] = -math.inf
        # the tokens that came are likely ones; every ninth place is padding
        pick = torch.randint(v, (n, 64), generator=g, device=dev)
        best = torch.gather(s["logits"], 1, pick).float().argmax(1)
        tokens = torch.gather(pick, 1, best[:, None])[:, 0].to(torch.int32)
        s["tokens"] = torch.where(torch.arange(n, device=dev) % 9 == 8, torch.full_like(tokens, -1), tokens)
        if own:
            s["logprob"], s["entropy"] = (torch.empty(n, device=dev) for _ in range(2))
            s["top_tokens"] = torch.empty((n, k), dtype=torch.int32, device=dev) if k else None
            s["top_logprobs"] = torch.empty((n, k), device=dev) if k else None
            s["job"] = trit.LogprobJob(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["top_tokens"],
                                       s["top_logprobs"])
        return s
    b, hq, hkv, d, dt = case["b"], case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    if case["op"] == "prompt":
        nq, nk = _queries(case)
        s["q_starts"], s["k_starts"] = _starts(nq, dev), _starts(nk, dev)
        s["q"] = rand(sum(nq), hq, d).mul_(1.5).to(dt)
        s["k"], s["v"] = (rand(sum(nk), hkv, d).to(dt) for _ in range(2))
        if own:
            s["out"] = torch.empty((sum(nq), hq, d), dtype=dt, device=dev)
            s["lse"] = torch.empty((sum(nq), hq), device=dev)
            s["job"] = trit.PromptJob(s["q"], s["k"], s["v"], s["out"], s["q_starts"], s["k_starts"], lse=s["lse"],
                                      scale=d ** -0.5)
        return s
    t = case["t"]
    pages, s["prefix_table"], s["table"], s["spare"] = _paged(case, g, dev)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    new = torch.tensor(_new(case), dtype=torch.int32, device=dev)
    s["new_lens"] = new if case["ragged"] and not case.get("packed") else None
    for x, mul in (("k", 0.3), ("v", 0.25)):       # steps of a usual spread, offsets near the middle
        s[x + "_codes"] = torch.randint(256, (pages, hkv, case["page"], d // 2), generator=g, device=dev, dtype=torch.uint8)
        step = mul * (1 + 0.2 * rand(pages, hkv, case["page"], d // GROUP).clamp(-3, 3))
        s[x + "_scale"] = torch.stack((step, step * (-7.5 + 0.3 * torch.rand(step.shape, generator=g, device=dev))), -1).half()
    batch = None
    if own:
        cache = trit.Kv4Cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        batch = trit.KvBatch(s["table"], s["lens"], t, new_lens=s["new_lens"], prefix_table=s["prefix_table"],
                             prefix_len=case.get("prefix", 0))
    if case["op"] == "cache":
        src, rows = DTYPES[case["src"]], (sum(_new(case)) if case["packed"] else b * t)
        s["starts"] = _starts(_new(case), dev) if case["packed"] else None
        s["k_starts"] = _starts(_lens(case), dev)
        s["q"], s["k"], s["v"] = (rand(rows, h, d).mul_(m).to(src) for h, m in ((hq, 3.0), (hkv, 3.0), (hkv, 0.7)))
        ang = torch.arange(case["own_max"], device=dev, dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["q_gain"] = 1 + 0.2 * rand(d) if case["norm"] else None
        if own:
            s["q_out"] = torch.zeros((rows, hq, d), dtype=dt, device=dev)
            total = sum(_lens(case))
            s["k_out"], s["v_out"] = (torch.empty((total, hkv, d), dtype=dt, device=dev) for _ in range(2))
            rope = trit.Rope(s["cos"], s["sin"], pairs=case["pairs"], q_gain=s["q_gain"], eps=1e-5)
            q_out = s["q_out"] if case["packed"] else s["q_out"].view(b, t, hq, d)
            s["job"] = trit.Append4Job(cache, batch, rope, s["q"], s["k"], s["v"], q_out, starts=s["starts"])
            s["read"] = trit.Read4Job(cache, batch, s["k_out"], s["v_out"], s["k_starts"])
    else:
        s["q"] = rand(b, t, hq, d).mul_(1.5).to(dt)
        if own:
            s["out"] = torch.empty((b, t, hq, d), dtype=dt, device=dev)
            s["lse"] = torch.empty((b, t, hq), device=dev)
            s["job"] = trit.Attn4Job(cache, batch, s["q"], s["out"], lse=s["lse"], scale=d ** -0.5)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import bit_plane_select_gb300 as trit
        if op == "prompt":
            trit.trit_attn_prompt(s["job"], s["err"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "cache":
            trit.trit_kv4_append(s["job"], s["err"])
            trit.trit_kv4_read(s["read"], s["err"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        if op == "attn4":
            trit.trit_attn_paged4(s["job"], s["err"])
            return {"out": s["out"], "lse": s["lse"]}
        trit.trit_logprobs(s["job"], s["err"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "top_tokens": s["top_tokens"],
                "top_logprobs": s["top_logprobs"]}
    return {"prompt": _prompt, "cache": _cache, "attn4": _attn4, "logprobs": _logprobs}[op](s)


# ---- the plain forms -----------------------------------------------------------


def _which(starts, total):
    """(sequence, place in it) of each packed row."""
    row = torch.arange(total, device=starts.device)
    b = torch.searchsorted(starts[1:], row.to(torch.int32), right=True)
    return b, row - starts.long()[b]


def _prompt(s):
    c = s["case"]
    nq, nk = (max(x) for x in _queries(c))
    b, hkv, d = c["b"], c["hkv"], c["d"]
    grp, dev = c["hq"] // hkv, s["q"].device
    qs, ks = s["q_starts"].long(), s["k_starts"].long()
    n, m = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    t, j = torch.arange(nq, device=dev), torch.arange(nk, device=dev)
    q = s["q"][(qs[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)].float() * (d ** -0.5)      # [b, nq, hq, d]
    k, v = (x[(ks[:-1, None] + j).clamp(max=x.shape[0] - 1)].permute(0, 2, 1, 3).float() for x in (s["k"], s["v"]))
    rows = q.reshape(b, nq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * nq, d)
    w = torch.matmul(rows, k.transpose(-1, -2)).reshape(b, hkv, grp, nq, nk)
    see = j[None, None, :] <= (t[None, :] + (m - n)[:, None])[:, :, None]
    w = w.masked_fill_(~see[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    e = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.reshape(b, hkv, grp * nq, nk), v).reshape(b, hkv, grp, nq, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (torch.log(total) + top)[..., 0]
    at = _which(s["q_starts"], s["q"].shape[0])
    out = out.permute(0, 3, 1, 2, 4).reshape(b, nq, c["hq"], d)[at]
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(b, nq, c["hq"])[at]}


def _rotated(x, gain, cos, sin, rot, pairs):
    x = x.float()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * gain
    cos, sin = cos[:, None, :], sin[:, None, :]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _quantised(x):
    """fp32 [..., d] -> codes [..., d] and (s, z) fp16 [..., d / 64, 2]."""
    x = x.unflatten(-1, (-1, GROUP)).clamp(-65504.0, 65504.0)
    low, high = x.amin(-1), x.amax(-1)
    step = ((high - low).double() / 15.0).float().half()
    z = low.half()
    inv = torch.where(step > 0, (1.0 / step.double()).float(), torch.zeros_like(low))
    c = torch.round((x - z.float()[..., None]) * inv[..., None]).clamp(0, 15)
    return c.flatten(-2), torch.stack((step, z), -1)


def _values(codes, scale):
    """What packed codes [..., d / 2] and (s, z) [..., d / 64, 2] stand for, fp32."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    f = scale.float()
    return (c * f[..., 0:1] + f[..., 1:2]).flatten(-2)


def _cache(s):
    c = s["case"]
    rows, t, page, dev = s["q"].shape[0], c["t"], c["page"], s["q"].device
    if c["packed"]:
        b, i = _which(s["starts"], rows)
        own_at = s["lens"].long()[b] - (s["starts"][1:] - s["starts"][:-1]).long()[b] + i
        there = torch.ones_like(b, dtype=torch.bool)
    else:
        row = torch.arange(rows, device=dev)
        b, i = row // t, row % t
        n = s["new_lens"].long()[b] if s["new_lens"] is not None else torch.full_like(b, t)
        own_at, there = s["lens"].long()[b] - n + i, i < n
    at = torch.where(there, own_at, torch.zeros_like(own_at))
    cos, sin = s["cos"][at], s["sin"][at]
    q = _rotated(s["q"], s["q_gain"], cos, sin, c["rot"], c["pairs"])
    q = torch.where(there[:, None, None], q, torch.zeros_like(q)).to(DTYPES[c["dtype"]])
    k = _rotated(s["k"], None, cos, sin, c["rot"], c["pairs"])
    # padding rows go to a page that no sequence has
    where = torch.where(there, s["table"].long()[b, at // page], s["spare"])
    for x, name in ((k, "k"), (s["v"].float(), "v")):
        codes, scale = _quantised(x)
        s[name + "_codes"][where, :, at % page] = (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8)
        s[name + "_scale"][where, :, at % page] = scale
    kb, j = _which(s["k_starts"], sum(_lens(c)))
    where, slot = s["table"].long()[kb, j // page], j % page
    k, v = (_values(s[x + "_codes"][where, :, slot], s[x + "_scale"][where, :, slot]).to(DTYPES[c["dtype"]])
            for x in ("k", "v"))
    return {"q": q, "k": k, "v": v}


def _attn4(s):
    c = s["case"]
    b, t, hkv, d, p = c["b"], c["t"], c["hkv"], c["d"], c["prefix"]
    grp, dev = c["hq"] // hkv, s["q"].device
    q = s["q"].float().reshape(b, t, hkv, grp, d) * (d ** -0.5)
    own_k, own_v = (_values(s[x + "_codes"][s["table"].long()], s[x + "_scale"][s["table"].long()])
                    .permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d) for x in ("k", "v"))
    rows = q.permute(0, 2, 1, 3, 4).reshape(b, hkv, t * grp, d)
    scores = torch.matmul(rows, own_k.transpose(-1, -2)).reshape(b, hkv, t, grp, -1)
    step = torch.arange(t, device=dev)[None, :]
    n = s["new_lens"][:, None] if s["new_lens"] is not None else torch.full_like(s["lens"][:, None], t)
    at, there = s["lens"][:, None] - n + step, step < n
    seen = torch.arange(scores.shape[-1], device=dev)[None, None, :] <= at[:, :, None]
    seen = (seen & there[:, :, None])[:, None, :, None, :]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if p:
        pre_k, pre_v = (_values(s[x + "_codes"][s["prefix_table"].long()], s[x + "_scale"][s["prefix_table"].long()])
                        .permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :p] for x in ("k", "v"))
        flat = q.permute(2, 0, 1, 3, 4).reshape(hkv, b * t * grp, d)
        pre = torch.matmul(flat, pre_k.transpose(-1, -2)).reshape(hkv, b, t, grp, p).transpose(0, 1)
        pre = pre.masked_fill(~there[:, None, :, None, None], -math.inf)
        top = torch.maximum(top, pre.amax(-1, keepdim=True))
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - base)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.reshape(b, hkv, t * grp, -1), own_v).reshape(b, hkv, t, grp, d)
    if p:
        e = torch.exp(pre - base)
        total = total + e.sum(-1, keepdim=True)
        o = torch.matmul(e.transpose(0, 1).reshape(hkv, b * t * grp, p), pre_v)
        out = out + o.reshape(hkv, b, t, grp, d).transpose(0, 1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (torch.log(total) + base)[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(b, t, c["hq"], d).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(b, t, c["hq"])}


def _logprobs(s):
    k, v = s["case"]["top"], s["case"]["vocab"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(1)
    mean = torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1) / total
    base = top[:, 0] + torch.log(total)
    tok = s["tokens"].long()
    given = torch.gather(d, 1, tok.clamp(min=0)[:, None])[:, 0] - torch.log(total)
    r = {"logprob": torch.where(tok < 0, torch.zeros_like(given), given), "entropy": torch.log(total) - mean,
         "top_tokens": None, "top_logprobs": None}
    if k:
        # one whole number per entry, in the order of its value and then of the lower index
        bits = (x + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 31) + (v - 1 - torch.arange(v, device=x.device))
        idx = torch.topk(key, k, 1).indices
        r["top_tokens"] = idx.to(torch.int32)
        r["top_logprobs"] = torch.gather(x, 1, idx) - base[:, None]
    return r


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"prompt": _exact_prompt, "cache": _exact_cache, "attn4": _exact_attn4, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_prompt(s):
    c = s["case"]
    nq, nk = _queries(c)
    grp, dev = c["hq"] // c["hkv"], s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    qa = ka = 0
    for n, m in zip(nq, nk):
        hidden = torch.arange(m, device=dev)[None, :] > torch.arange(n, device=dev)[:, None] + (m - n)
        for h in range(c["hq"]):
            w = s["q"][qa:qa + n, h].double() @ s["k"][ka:ka + m, h // grp].double().T / math.sqrt(c["d"])
            w[hidden] = -math.inf
            top = torch.logsumexp(w, -1)
            out[qa:qa + n, h] = torch.exp(w - top[:, None]) @ s["v"][ka:ka + m, h // grp].double()
            lse[qa:qa + n, h] = top
        qa, ka = qa + n, ka + m
    return {"out": out, "lse": lse}


def _fp32(x):
    return x.float().double()


def _turn(x, cos, sin, rot, pairs, rounded):
    """x [rows, heads, d] turned by the rows' angles; `rounded`: to fp32 after each operation."""
    r = _fp32 if rounded else (lambda v: v)
    y = x.clone()
    first = list(range(0, rot, 2)) if pairs else list(range(rot // 2))
    second = list(range(1, rot, 2)) if pairs else list(range(rot // 2, rot))
    a, b, cos, sin = x[..., first], x[..., second], cos[:, None, :], sin[:, None, :]
    y[..., first] = r(r(a * cos) - r(b * sin))
    y[..., second] = r(r(b * cos) + r(a * sin))
    return y


def _exact_stored(x):
    """What a vector [rows, heads, d] of fp32 values stands for once it is held in 4 bits."""
    y = torch.empty_like(x)
    for at in range(0, x.shape[-1], GROUP):
        part = x[..., at:at + GROUP].clamp(-65504.0, 65504.0)
        low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        step = _fp32(_fp32(high - low) / 15.0).half().double()
        z = low.half().double()
        c = _fp32(_fp32(part - z) * _fp32(1.0 / step)).round().clamp(0, 15)
        y[..., at:at + GROUP] = torch.where(step > 0, c * step + z, z)
    return y


def _unpacked(codes, scale):
    """Packed codes and (s, z) as 64-bit values."""
    y = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
    y[..., 0::2], y[..., 1::2] = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    f = scale.double().repeat_interleave(GROUP, -2)
    return y * f[..., 0] + f[..., 1]


def _exact_cache(s):
    c = s["case"]
    lens, new, page, dev = _lens(c), _new(c), c["page"], s["q"].device
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    made = {"k": [], "v": []}
    at = 0
    for b in range(c["b"]):
        n, first = new[b], at if c["packed"] else b * c["t"]
        at += n
        i = torch.arange(lens[b], device=dev)
        where = s["table"][b].long()[i // page]
        cos, sin = s["cos"][i[lens[b] - n:]].double(), s["sin"][i[lens[b] - n:]].double()
        x = s["q"][first:first + n].double()
        if s["q_gain"] is not None:
            x = x * (x.square().mean(-1, keepdim=True) + 1e-5) ** -0.5 * s["q_gain"].double()
        q[first:first + n] = _turn(x, cos, sin, c["rot"], c["pairs"], False)
        fresh = {"k": _turn(s["k"][first:first + n].double(), cos, sin, c["rot"], c["pairs"], True),
                 "v": s["v"][first:first + n].double()}
        for name in ("k", "v"):
            old = _unpacked(s[name + "_codes"][where, :, i % page], s[name + "_scale"][where, :, i % page])
            old[lens[b] - n:] = _exact_stored(fresh[name])
            made[name].append(old)
    return {"q": q, "k": torch.cat(made["k"]), "v": torch.cat(made["v"])}


def _exact_attn4(s):
    c = s["case"]
    lens, new, p, page, hkv = _lens(c), _new(c), c["prefix"], c["page"], c["hkv"]
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=dev)
    i = torch.arange(p, device=dev)
    where = s["prefix_table"].long()[i // page] if p else i
    pk, pv = (_unpacked(s[x + "_codes"][where, :, i % page], s[x + "_scale"][where, :, i % page]).transpose(0, 1)
              for x in ("k", "v"))
    for b in range(c["b"]):
        j = torch.arange(lens[b], device=dev)
        where = s["table"][b].long()[j // page]
        k, v = (torch.cat((pre, _unpacked(s[x + "_codes"][where, :, j % page],
                                          s[x + "_scale"][where, :, j % page]).transpose(0, 1)), 1)
                for pre, x in ((pk, "k"), (pv, "v")))
        for t in range(new[b]):
            seen = p + lens[b] - new[b] + t + 1
            rows = s["q"][b, t].double().reshape(hkv, -1, c["d"])
            w = torch.bmm(rows, k[:, :seen].transpose(1, 2)) / math.sqrt(c["d"])
            top = torch.logsumexp(w, -1)
            out[b, t] = torch.bmm(torch.exp(w - top[..., None]), v[:, :seen]).reshape(c["hq"], c["d"])
            lse[b, t] = top.reshape(-1)
    return {"out": out, "lse": lse}


def _exact_logprobs(s):
    n, v = s["logits"].shape
    k = s["case"]["top"]
    dev = s["logits"].device
    given, entropy = (torch.zeros(n, dtype=torch.float64, device=dev) for _ in range(2))
    ids = torch.zeros((n, k), dtype=torch.int32, device=dev)
    best = torch.zeros((n, k), dtype=torch.float64, device=dev)
    step = max(1, (1 << 25) // v)
    for i in range(0, n, step):
        logp = torch.log_softmax(s["logits"][i:i + step].double(), -1)
        tok = s["tokens"][i:i + step].long()
        given[i:i + step] = torch.where(tok < 0, 0.0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0])
        entropy[i:i + step] = -(logp.exp() * logp.clamp(min=-1e300)).sum(-1)
        left = s["logits"][i:i + step].double()
        for m in range(k):
            ids[i:i + step, m] = left.argmax(-1).to(torch.int32)
            best[i:i + step, m] = logp.gather(1, ids[i:i + step, m:m + 1].long())[:, 0]
            left.scatter_(1, ids[i:i + step, m:m + 1].long(), -math.inf)
    return {"logprob": given, "entropy": entropy, "top_tokens": ids if k else None, "top_logprobs": best if k else None}


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    if case["op"] == "logprobs":
        n, v, e = case["rows"], case["vocab"], (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": n * v * e + n * (12 + 8 * case["top"]), "flops": 4.0 * n * v}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "prompt":
        nq, nk = _queries(case)
        pairs = sum(n * m - n * (n - 1) / 2 for n, m in zip(nq, nk))
        return {"bytes": sum(nq) * hq * (d * 4 + 4) + sum(nk) * hkv * d * 4, "flops": 4.0 * pairs * hq * d}
    lens, n = _lens(case), sum(_new(case))
    vector = d // 2 + 4 * d // GROUP                 # bytes of a key or value of one head
    if case["op"] == "cache":
        e = 4 if case["src"] == "fp32" else 2
        old = sum(lens) - n
        # the new rows in, the queries out, the new vectors stored, the old ones read, every value out
        return {"bytes": n * ((hq + 2 * hkv) * d * e + hq * d * 2 + case["rot"] * 4) + (n + old) * 2 * hkv * vector +
                sum(lens) * 2 * hkv * d * 2, "flops": 8.0 * n * (hq + 2 * hkv) * d}
    p = case["prefix"]
    keys = p + sum(lens)
    pairs = sum(m * p + sum(lens[i] - m + 1 + k for k in range(m)) for i, m in enumerate(_new(case)))
    return {"bytes": keys * hkv * 2 * vector + n * hq * d * 4 + n * hq * 4, "flops": 4.0 * pairs * hq * d}
