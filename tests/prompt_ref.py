"""Plain implementations of the operators of prompts, of the 4-bit cache and of scoring,
and caches to test them on.  Shared by the GPU tests; CPU tensors only."""
import math

import torch

GROUP = 64


def quantised(x):
    """fp32 [..., D] -> codes [..., D] (whole numbers) and (s, z) fp16 [..., D / 64, 2], every
    operation rounded to fp32 as the format says."""
    x = x.float().unflatten(-1, (-1, GROUP))
    bad = ~x.isfinite().all(-1)
    x = x.nan_to_num(0, 0, 0).clamp(-65504.0, 65504.0)
    low, high = x.amin(-1), x.amax(-1)
    s = ((high - low).double() / 15.0).float().half()
    z = low.half()
    inv = torch.where(s > 0, (1.0 / s.double()).float(), torch.zeros_like(low))
    c = torch.round((x - z.float()[..., None]) * inv[..., None]).clamp(0, 15)
    s = torch.where(bad, torch.zeros_like(s), s)
    z = torch.where(bad, torch.full_like(z, math.nan), z)
    c = torch.where(bad[..., None], torch.zeros_like(c), c)
    return c.flatten(-2).to(torch.uint8), torch.stack((s, z), -1)


def pack(c):
    return c[..., 0::2] + 16 * c[..., 1::2]


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def values(codes, scale):
    """Packed codes and (s, z) -> what they stand for, in 64 bits (exactly)."""
    c = unpack(codes).unflatten(-1, (-1, GROUP)).double()
    f = scale.double()
    return (c * f[..., 0:1] + f[..., 1:2]).flatten(-2)


def random_cache(gen, pages, heads, page, D, nhd=False, spread=0.3):
    """Four CPU tensors of a cache of random codes; nhd: laid out [pages, page, heads, ...]."""
    made = []
    for _ in range(2):
        shape = (pages, page, heads) if nhd else (pages, heads, page)
        codes = torch.randint(256, shape + (D // 2,), generator=gen, dtype=torch.uint8)
        s = spread * (1 + 0.2 * torch.randn(shape + (D // GROUP,), generator=gen).clamp(-3, 3))
        z = s * (-7.5 + torch.randn(s.shape, generator=gen))
        made.append((codes, torch.stack((s, z), -1).half()))
    four = [made[0][0], made[1][0], made[0][1], made[1][1]]
    return [x.transpose(1, 2) for x in four] if nhd else four


def on_gpu(x):
    """The same layout on the GPU."""
    return x.cuda() if x.is_contiguous() else x.transpose(1, 2).cuda().transpose(1, 2)


def rotate32(x, cos, sin, rot, pairs):
    """fp32 [..., D] turned by one row of the tables, each operation rounded to fp32."""
    y = x.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
        y[..., a] = x[..., a] * cos[j] - x[..., b] * sin[j]
        y[..., b] = x[..., b] * cos[j] + x[..., a] * sin[j]
    return y


def causal(q, k, v, scale):
    """q [nq, Hq, D], k and v [nk, H, D] in 64 bits, the queries the last of the keys' tokens ->
    out [nq, Hq, D], lse [nq, Hq], and sum of softmax |v| (a scale for rounding)."""
    nq, hq, D = q.shape
    nk, h = k.shape[:2]
    g = hq // h
    out, mag = (torch.zeros(nq, hq, D, dtype=torch.float64) for _ in range(2))
    lse = torch.full((nq, hq), -math.inf, dtype=torch.float64)
    see = torch.arange(nk)[None, :] <= torch.arange(nq)[:, None] + (nk - nq)
    some = see.any(1)
    if not bool(some.any()):
        return out, lse, mag
    for i in range(hq):
        w = (q[some, i] @ k[:, i // g].T) * scale
        w = torch.where(see[some], w, torch.full_like(w, -math.inf))
        lse[some, i] = torch.logsumexp(w, 1)
        p = torch.exp(w - lse[some, i][:, None])
        out[some, i] = p @ v[:, i // g]
        mag[some, i] = p @ v[:, i // g].abs()
    return out, lse, mag


def scored(x, tokens, n):
    """One row at a time in 64 bits: (logprob, entropy, top tokens, top logprobs)."""
    rows, V = x.shape
    given, entropy = (torch.zeros(rows, dtype=torch.float64) for _ in range(2))
    ids, best = torch.full((rows, n), -1, dtype=torch.int32), torch.full((rows, n), -math.inf, dtype=torch.float64)
    for r in range(rows):
        y = x[r].double()
        t = int(tokens[r])
        if bool(y.isnan().any()) or bool((y == math.inf).any()):
            given[r], entropy[r], best[r] = (0.0 if t == -1 else math.nan), math.nan, math.nan
            if t < -1 or t >= V:
                given[r] = -math.inf
            continue
        some = y > -math.inf
        if not bool(some.any()):
            given[r] = 0.0 if t == -1 else -math.inf
            continue
        m = y.max()
        d = y[some] - m
        l = torch.exp(d).sum()
        given[r] = 0.0 if t == -1 else (float(y[t] - m - torch.log(l)) if 0 <= t < V else -math.inf)
        entropy[r] = torch.log(l) - (torch.exp(d) * d).sum() / l
        order = sorted(((-float(v), i) for i, v in enumerate(y.tolist()) if v > -math.inf))[:n]
        for j, (v, i) in enumerate(order):
            ids[r, j], best[r, j] = i, (-v - float(m)) - float(torch.log(l))
    return given, entropy, ids, best
