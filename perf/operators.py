"""The serving operators' cases: appending to a paged cache, attention over a
shared prefix and the sequences' own pages, and verification of drafted tokens.

A case's "op" says which: "append", "attn" or "verify".  `run` computes the
plain form in 32 bits with elementary torch operations, or, where `own` is
true, calls this package's kernels.  `exact` is the same from the definitions
in 64 bits, one sequence at a time.

Sizes: 20 query heads over 5 key heads of 128 columns are the framework's
layer (q 2560, k and v 640 rows); the other head layouts are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    a = {"op": "append", "hq": 20, "hkv": 5, "d": 128, "rot": 128, "page": 64, "dtype": "bf16",
         "src": "fp32", "norm": False, "pairs": False, "ragged": False, "prefix": 0}
    t = {"op": "attn", "hq": 20, "hkv": 5, "d": 128, "page": 64, "dtype": "bf16", "ragged": False}
    v = {"op": "verify", "dtype": "fp32", "ragged": False}
    return [
        # one token of one sequence between two products of a decode step: latency
        dict(a, name="append-one-token", b=1, t=1, own_min=700, own_max=700),
        # a ragged batch of drafted tokens, half heads, partial rotation of pairs, head norms
        dict(a, name="append-drafts", b=61, t=6, own_min=9, own_max=2100, hq=24, hkv=8, d=64, rot=48,
             page=16, dtype="fp16", norm=True, pairs=True, ragged=True, prefix=1003),
        # a chunk of prompt of four sequences, head norms on, q k v straight from the products
        dict(a, name="append-prefill", b=4, t=8192, own_min=8192, own_max=12000, norm=True),
        # one short conversation, one token: latency
        dict(t, name="attn-one-short", b=1, t=1, prefix=0, own_min=700, own_max=700),
        # two long documents, one token each: few rows over a long axis
        dict(t, name="attn-two-long", b=2, t=1, prefix=0, own_min=90000, own_max=131001),
        # a usual batch behind one system prompt
        dict(t, name="attn-batch", b=32, t=1, prefix=4096, own_min=33, own_max=900),
        # drafted tokens of a batch, verified in one pass, ragged, odd prefix, 16-token pages
        dict(t, name="attn-drafts", b=24, t=5, prefix=8005, own_min=6, own_max=1500, page=16, ragged=True),
        # half-width heads in fp16, no grouping to speak of
        dict(t, name="attn-half-heads", b=96, t=1, hq=16, hkv=8, d=64, prefix=6000, own_min=1, own_max=1300,
             page=32, dtype="fp16"),
        # the largest: a full batch behind a long shared document
        dict(t, name="attn-full-batch", b=256, t=1, prefix=32768, own_min=60, own_max=1600),
        # four drafted tokens of one sequence: latency
        dict(v, name="verify-one", b=1, t=4, vocab=32000, alpha=0.8),
        # a usual batch, odd vocabulary
        dict(v, name="verify-batch", b=24, t=5, vocab=50257, alpha=0.75, ragged=True),
        # the largest batch and vocabulary
        dict(v, name="verify-full-batch", b=192, t=8, vocab=131072, alpha=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "verify"])
    dtype = rng.choice(["bf16", "fp16"])
    hq, hkv, d = rng.choice([(20, 5, 128), (32, 8, 128), (16, 8, 64), (24, 8, 64), (8, 1, 128), (7, 7, 64)])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        b = _log(rng, 1, 128)
        t = min(_log(rng, 1, 4096), max(1, 16384 // b))
        lo = t + rng.randrange(0, 700)
        return {"op": op, "b": b, "t": t, "own_min": lo, "own_max": lo + rng.randrange(0, 900), "hq": hq, "hkv": hkv,
                "d": d, "rot": rng.choice([d, d, d // 2, d - 16]), "page": page, "dtype": dtype,
                "src": rng.choice(["fp32", dtype]), "norm": rng.random() < 0.5, "pairs": rng.random() < 0.3,
                "ragged": rng.random() < 0.4, "prefix": rng.choice([0, _log(rng, 1, 30000)])}
    if op == "attn":
        b = _log(rng, 1, 200)
        t = rng.choice([1, 1, 1, 2, 3, 5, 8])
        hi = max(t, min(_log(rng, 16, 120000), 300000 // (b * t) + t))
        # (b t) prefix hq d within the largest listed case
        prefix = rng.choice([0, _log(rng, 64, 32768)])
        prefix = min(prefix, 256 * 32768 * 20 * 128 // (2 * b * t * hq * d))
        return {"op": op, "b": b, "t": t, "prefix": prefix, "own_min": max(t, hi // rng.choice([1, 2, 10])),
                "own_max": hi, "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype,
                "ragged": rng.random() < 0.4}
    b = _log(rng, 1, 160)
    return {"op": op, "b": b, "t": rng.randrange(1, 9), "vocab": _log(rng, 2000, 131072),
            "alpha": round(rng.uniform(0.3, 0.95), 3), "dtype": rng.choice(["fp32", "fp32", "bf16"]),
            "ragged": rng.random() < 0.4}


def _lens(case):
    """Own lengths of the sequences, from the case alone (work() counts them)."""
    b, lo, hi = case["b"], case["own_min"], case["own_max"]
    return [lo + (hi - lo) * ((37 * i + 11) % max(2, b) + 1) // max(2, b) for i in range(b)] if b > 1 else [hi]


def _new(case):
    """Valid new tokens of the sequences: all t, or ragged 1..t."""
    b, t = case["b"], case["t"]
    return [1 + ((i + 1) * 2654435761 >> 9) % t for i in range(b)] if case["ragged"] else [t] * b


def _paged(case, g, dev):
    """Page ids of the prefix and the sequences, scattered over the cache."""
    lens, page = _lens(case), case["page"]
    need = [-(-n // page) for n in lens]
    npre = -(-case["prefix"] // page)
    pages = sum(need) + npre + 3
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((case["b"], max(need)), dtype=torch.int32, device=dev)
    col = torch.arange(max(need), device=dev)
    first = torch.tensor([npre + sum(need[:i]) for i in range(len(need))], device=dev)
    n = torch.tensor(need, device=dev)
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.where(col[None, :] < n[:, None], ids[at], table)
    return pages, ids[:npre].contiguous(), table.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    rand = lambda *n: torch.randn(*n, generator=g, device=dev)  # noqa: E731
    b, t = case["b"], case["t"]
    new = torch.tensor(_new(case), dtype=torch.int32, device=dev)
    s["new_lens"] = new if case["ragged"] else None
    if case["op"] == "verify":
        v, dt = case["vocab"], DTYPES[case["dtype"]]
        s["p"] = torch.empty((b, t + 1, v), dtype=dt, device=dev)
        s["q"] = torch.empty((b, t, v), dtype=dt, device=dev)
        for i in range(b):  # peaked rows; the draft is right about alpha of the mass
            p = torch.softmax(2.5 * rand(t + 1, v), -1)
            r = torch.softmax(2.5 * rand(t, v), -1)
            s["p"][i] = p.to(dt)
            s["q"][i] = (case["alpha"] * p[:t] + (1 - case["alpha"]) * r).to(dt)
        s["draft"] = torch.multinomial(s["q"].float().reshape(b * t, v), 1, generator=g).reshape(b, t).to(torch.int32)
        s["u"] = torch.rand((b, t), generator=g, device=dev)
        s["race"] = torch.empty((b, v), device=dev).exponential_(generator=g)
        if own:
            import bit_plane_select_gb300 as trit
            s["tokens"] = torch.empty((b, t + 1), dtype=torch.int32, device=dev)
            s["accepted"] = torch.empty(b, dtype=torch.int32, device=dev)
            s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
            s["job"] = trit.VerifyJob(s["p"], s["q"], s["draft"], s["u"], s["race"], s["tokens"], s["accepted"],
                                      n_draft=s["new_lens"])
        return s
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    pages, s["prefix_table"], s["table"] = _paged(case, g, dev)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    s["k_cache"] = rand(pages, hkv, case["page"], d).to(dt)
    s["v_cache"] = rand(pages, hkv, case["page"], d).to(dt)
    if case["op"] == "append":
        src = DTYPES[case["src"]]
        s["q"], s["k"], s["v"] = (rand(b, t, h, d).mul_(m).to(src) for h, m in ((hq, 3.0), (hkv, 3.0), (hkv, 0.7)))
        top = case["prefix"] + case["own_max"]
        ang = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["q_gain"], s["k_gain"] = (1 + 0.2 * rand(d), 1 + 0.2 * rand(d)) if case["norm"] else (None, None)
    else:
        s["q"] = rand(b, t, hq, d).mul_(1.5).to(dt)
    if own:
        import bit_plane_select_gb300 as trit
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
        cache = trit.KvCache(s["k_cache"], s["v_cache"])
        batch = trit.KvBatch(s["table"], s["lens"], t, new_lens=s["new_lens"], prefix_table=s["prefix_table"],
                             prefix_len=case["prefix"])
        if case["op"] == "append":
            s["q_out"] = torch.zeros((b, t, hq, d), dtype=dt, device=dev)
            rope = trit.Rope(s["cos"], s["sin"], pairs=case["pairs"], q_gain=s["q_gain"], k_gain=s["k_gain"], eps=1e-5)
            s["job"] = trit.AppendJob(cache, batch, rope, s["q"], s["k"], s["v"], s["q_out"])
        else:
            s["out"] = torch.empty((b, t, hq, d), dtype=dt, device=dev)
            s["lse"] = torch.empty((b, t, hq), dtype=torch.float32, device=dev)
            s["job"] = trit.AttnJob(cache, batch, s["q"], s["out"], lse=s["lse"], scale=d ** -0.5)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import bit_plane_select_gb300 as trit
        if op == "append":
            trit.trit_kv_append(s["job"], s["err"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "attn":
            trit.trit_attn_paged(s["job"], s["err"])
            return {"out": s["out"], "lse": s["lse"]}
        trit.trit_draft_verify(s["job"], s["err"])
        return {"tokens": s["tokens"], "accepted": s["accepted"]}
    return {"append": _append, "attn": _attn, "verify": _verify}[op](s)


# ---- the plain forms -----------------------------------------------------------


def _positions(s):
    """[b, t]: the own index of each new token, and which are there."""
    c = s["case"]
    t = torch.arange(c["t"], device=s["lens"].device)[None, :]
    n = s["new_lens"][:, None] if s["new_lens"] is not None else torch.full_like(s["lens"][:, None], c["t"])
    return s["lens"][:, None] - n + t, t < n


def _rotated(x, gain, cos, sin, rot, pairs):
    x = x.float()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * gain
    cos, sin = cos[:, :, None, :], sin[:, :, None, :]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    at, there = _positions(s)
    at = torch.where(there, at, torch.zeros_like(at)).long()
    pos = at + c["prefix"]
    cos, sin = s["cos"][pos], s["sin"][pos]
    dt = s["k_cache"].dtype
    q = _rotated(s["q"], s["q_gain"], cos, sin, c["rot"], c["pairs"])
    k = _rotated(s["k"], s["k_gain"], cos, sin, c["rot"], c["pairs"])
    q = torch.where(there[:, :, None, None], q, torch.zeros_like(q)).to(dt)
    page = torch.gather(s["table"].long(), 1, at // c["page"])
    ok = there.reshape(-1)
    page, slot = page.reshape(-1)[ok], (at % c["page"]).reshape(-1)[ok]
    s["k_cache"][page, :, slot] = k.flatten(0, 1)[ok].to(dt)
    s["v_cache"][page, :, slot] = s["v"].flatten(0, 1)[ok].to(dt)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn(s):
    c = s["case"]
    b, t, hkv, d, p = c["b"], c["t"], c["hkv"], c["d"], c["prefix"]
    grp = c["hq"] // hkv
    q = s["q"].float().reshape(b, t, hkv, grp, d) * (d ** -0.5)
    own_k, own_v = (x[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d).float()
                    for x in (s["k_cache"], s["v_cache"]))
    rows = q.permute(0, 2, 1, 3, 4).reshape(b, hkv, t * grp, d)
    scores = torch.matmul(rows, own_k.transpose(-1, -2)).reshape(b, hkv, t, grp, -1)
    at, there = _positions(s)
    seen = torch.arange(scores.shape[-1], device=q.device)[None, None, :] <= at[:, :, None]
    seen = (seen & there[:, :, None])[:, None, :, None, :]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if p:
        pre_k, pre_v = (x[s["prefix_table"].long()].permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :p].float()
                        for x in (s["k_cache"], s["v_cache"]))
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


def _verify(s):
    b, t, v = s["q"].shape
    seq = torch.arange(b, device=s["q"].device)
    step = torch.arange(t, device=s["q"].device)[None, :]
    n = s["new_lens"].long() if s["new_lens"] is not None else torch.full_like(seq, t)
    x = s["draft"].long()[:, :, None]
    px = torch.gather(s["p"][:, :t], 2, x)[..., 0].float()
    qx = torch.gather(s["q"], 2, x)[..., 0].float()
    fine = (s["u"] * qx < px) & (step < n[:, None])
    took = fine.long().cumprod(1).sum(1)
    p = s["p"][seq, took].float()
    q = s["q"][seq, took.clamp(max=t - 1)].float()
    left = torch.where((took < n)[:, None], p - q, p)
    left = torch.where((left > 0).any(1, keepdim=True), left, p)
    score = torch.where(left > 0, left / s["race"], torch.full_like(left, -1.0))
    token = torch.argmax(score, 1).to(torch.int32)
    tokens = torch.full((b, t + 1), -1, dtype=torch.int32, device=s["q"].device)
    tokens[:, :t] = torch.where(step < took[:, None], s["draft"], tokens[:, :t])
    tokens[seq, took] = token
    return {"tokens": tokens, "accepted": took.to(torch.int32)}


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify}[case["op"]](s)


def _turn(x, angle_cos, angle_sin, rot, pairs):
    """x [tokens, heads, d] as complex numbers times cos + i sin."""
    y = x.clone()
    first = list(range(0, rot, 2)) if pairs else list(range(rot // 2))
    second = list(range(1, rot, 2)) if pairs else list(range(rot // 2, rot))
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_cos, angle_sin)[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(s):
    c = s["case"]
    lens, new = _lens(c), _new(c)
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b in range(c["b"]):
        n = new[b]
        i = torch.arange(lens[b] - n, lens[b], device=q.device)
        cos, sin = s["cos"][i + c["prefix"]].double(), s["sin"][i + c["prefix"]].double()
        made = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            x = x[b, :n].double()
            if gain is not None:
                x = x * (x.square().mean(-1, keepdim=True) + 1e-5) ** -0.5 * gain.double()
            made.append(_turn(x, cos, sin, c["rot"], c["pairs"]))
        q[b, :n] = made[0]
        page = s["table"][b].long()[i // c["page"]]
        kc[page, :, i % c["page"]] = made[1]
        vc[page, :, i % c["page"]] = s["v"][b, :n].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_attn(s):
    c = s["case"]
    lens, new, p, page, hkv = _lens(c), _new(c), c["prefix"], c["page"], c["hkv"]
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=dev)
    i = torch.arange(p, device=dev)
    where = s["prefix_table"].long()[i // page] if p else i
    pk, pv = (x[where, :, i % page].double().transpose(0, 1) for x in (s["k_cache"], s["v_cache"]))
    for b in range(c["b"]):
        j = torch.arange(lens[b], device=dev)
        where = s["table"][b].long()[j // page]
        k, v = (torch.cat((pre, x[where, :, j % page].double().transpose(0, 1)), 1)
                for pre, x in ((pk, s["k_cache"]), (pv, s["v_cache"])))
        for t in range(new[b]):
            seen = p + lens[b] - new[b] + t + 1
            rows = s["q"][b, t].double().reshape(hkv, -1, c["d"])
            w = torch.bmm(rows, k[:, :seen].transpose(1, 2)) / math.sqrt(c["d"])
            top = torch.logsumexp(w, -1)
            out[b, t] = torch.bmm(torch.exp(w - top[..., None]), v[:, :seen]).reshape(c["hq"], c["d"])
            lse[b, t] = top.reshape(-1)
    return {"out": out, "lse": lse}


def _exact_verify(s):
    b, t, v = s["q"].shape
    n = _new(s["case"])
    tokens = torch.full((b, t + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(b, dtype=torch.int32)
    draft, u = s["draft"].cpu(), s["u"].double().cpu()
    for i in range(b):
        k = 0
        while k < n[i]:
            x = int(draft[i, k])
            if not float(u[i, k]) * float(s["q"][i, k, x]) < float(s["p"][i, k, x]):
                break
            tokens[i, k] = x
            k += 1
        left = s["p"][i, k].double()
        if k < n[i]:
            less = (left - s["q"][i, k].double()).clamp(min=0)
            left = less if bool((less > 0).any()) else left
        tokens[i, k] = int(torch.argmin(torch.where(left > 0, s["race"][i].double() / left, math.inf)))
        accepted[i] = k
    return {"tokens": tokens, "accepted": accepted}


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    b, t, new = case["b"], case["t"], _new(case)
    if case["op"] == "verify":
        e, v = (2 if case["dtype"] == "bf16" else 4), case["vocab"]
        rejected = sum(1 - case["alpha"] ** n for n in new)  # the share of sequences that read q's row too
        return {"bytes": b * v * (e + 4) + rejected * v * e + sum(new) * (2 * e + 8) + b * (4 * t + 8),
                "flops": 2.0 * b * v}
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], sum(new)
    if case["op"] == "append":
        e = 4 if case["src"] == "fp32" else 2
        heads = hq + 2 * hkv
        return {"bytes": n * heads * d * (e + 2) + n * case["rot"] * 4, "flops": n * (hq + hkv) * d * (6.0 if case["norm"] else 3.0)}
    lens, p = _lens(case), case["prefix"]
    keys = p + sum(lens)
    pairs = sum(m * p + sum(lens[i] - m + 1 + k for k in range(m)) for i, m in enumerate(new))
    return {"bytes": keys * hkv * d * 4 + n * hq * d * 4 + n * hq * 4, "flops": 4.0 * pairs * hq * d}
