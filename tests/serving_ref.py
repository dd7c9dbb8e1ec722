"""Plain 64-bit implementations of the serving operators, token by token, and
paged batches to test them on.  Shared by the GPU tests; CPU tensors only."""
import math

import torch

NAN = float("nan")


def make_batch(gen, lens, T, page_size, prefix_len=0, extra_cols=2):
    """Scattered page ids: (pages, prefix_table, table).  Unused table entries
    name page 0, which belongs to nobody."""
    need = [-(-n // page_size) for n in lens]
    npre = -(-prefix_len // page_size)
    pages = 1 + npre + sum(need) + 2
    ids = (1 + torch.randperm(pages - 1, generator=gen)).to(torch.int32)
    table = torch.zeros((len(lens), max(need + [1]) + extra_cols), dtype=torch.int32)
    at = npre
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return pages, ids[:npre].contiguous(), table


def slots(table_row, n, page_size):
    i = torch.arange(n)
    return table_row.long()[i // page_size], i % page_size


def rotate(x, cos, sin, rot, pairs):
    """One head vector (64 bits) turned by one row of the tables."""
    y = x.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
        y[..., a] = x[..., a] * cos[j] - x[..., b] * sin[j]
        y[..., b] = x[..., b] * cos[j] + x[..., a] * sin[j]
    return y


def normed(x, gain, eps):
    return x if gain is None else x / math.sqrt(float((x * x).mean(-1)) + eps) * gain


def attend(q, keys, vals, scale):
    """q [Hq, D], keys and vals [n, Hkv, D] in 64 bits -> out [Hq, D], lse [Hq]."""
    hq, d = q.shape
    n, hkv = keys.shape[0], keys.shape[1] if keys.dim() == 3 else 1
    if n == 0:
        return torch.zeros(hq, d, dtype=torch.float64), torch.full((hq,), -math.inf, dtype=torch.float64)
    out, lse = [], []
    for h in range(hq):
        hk = h // (hq // hkv)
        s = (keys[:, hk] @ q[h]) * scale
        lse.append(torch.logsumexp(s, 0))
        out.append(torch.exp(s - lse[-1]) @ vals[:, hk])
    return torch.stack(out), torch.stack(lse)


def verify(p, q, draft, u, race, n):
    """One sequence -> (tokens, accepted), in fp32 where the definition rounds."""
    T = draft.shape[0]
    tokens, k = [-1] * (T + 1), 0
    while k < n:
        x = int(draft[k])
        if not 0 <= x < q.shape[1] or not float((u[k] * q[k, x].float())) < float(p[k, x].float()):
            break
        tokens[k] = x
        k += 1
    r = p[k].float() - q[k].float() if k < n else p[k].float()
    if not bool((r > 0).any()):
        r = p[k].float()
    score = r / race
    ok = (r > 0) & (score >= 0)
    if bool(ok.any()):
        score = torch.where(ok, score, torch.full_like(score, -1.0))
        tokens[k] = int((score == score.max()).nonzero()[0])
    return tokens, k
