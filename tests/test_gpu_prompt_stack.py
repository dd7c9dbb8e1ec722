"""Prompts, the 4-bit cache and scoring together, as a user runs them: ServedStack with
cache_bits=4 and examples/score_prompts.py.

The products are exact, so a token's keys of the first layer do not depend on how its prompt came
in: whole, in turns, or token by token, the first layer's cache is the same bit by bit.  Every
step's attention is compared with 64-bit softmax attention over the queries and the cache's
values as they lie on the device, with the bounds of test_gpu_attn_prompt (whose keys
and values are the cache's, rounded once to 16 bits) and test_gpu_attn4 for fp32 outputs, the
scores' error taken from the step's own sizes."""
import importlib.util
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
from test_gpu_attn_paged import BF, HF, UNIT, t  # noqa: E402,F401
from test_gpu_served_stack_exact import layer  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
K, D, HQ, HK, PAGE = 192, 64, 4, 2, 16


def stack_of(t, dt, pages):  # noqa: F811
    from bit_plane_select_gb300.stack import ServedStack
    ang = torch.arange(400, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return ServedStack([layer(9), layer(10)], D, t.Rope(ang.cos().float().cuda(), ang.sin().float().cuda()), pages, PAGE,
                       dtype=dt, cache_bits=4)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def starts(n, first=0):
    return torch.tensor([first] + list(n), dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def cached(L, row, n):
    """Keys and values [n, HK, D] of a layer that a table row names, in 64 bits."""
    c = L["cache"]
    at = ref.slots(row, n, PAGE)
    return [pr.values(x.cpu(), s.cpu()).permute(0, 2, 1, 3)[at] for x, s in ((c.k, c.k_scale), (c.v, c.v_scale))]


def attends_right(got, q, k, v, dt, rounded):
    """got, q [n, HQ, D] of the last n tokens of k and v; rounded: keys and values in 16 bits."""
    q, got = q.double().cpu(), got.double().cpu()
    if rounded:
        k, v = (x.float().to(dt).double() for x in (k, v))
    # scores: D products and sums in fp32 of scale sum |q| (15 s + |z|) <= 3 scale sum |q| max |k|
    e = 3 * (D + 8) * 2.0 ** -24 * float(q.abs().sum(-1).max() * k.abs().max()) * D ** -0.5
    assert e < 2.0 ** -8        # (or the test would say little)
    want, _, mag = pr.causal(q, k, v, D ** -0.5)
    size = mag if rounded else mag + 2 * float(v.abs().max())      # |s c| + |z| <= |v| + 2 |z|
    w = UNIT[dt] if rounded else 2.0 ** -11
    return bool(((got - want).abs() <= (w + 2 * e + 2.0 ** -12) * size + 2.0 ** -16).all())


@pytest.mark.parametrize("dt", [BF, HF])
def test_whole_in_turns_and_by_token(t, dt):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    total, B = [70, 1, 150], 3
    pages, _, table = ref.make_batch(g, total, 1, PAGE)
    rows = [torch.randn(n, K, generator=g) for n in total]
    lens = ints(0, 0, 0)

    def go(stack, new, T, slack=2):
        """The next new[b] tokens of each sequence, packed, with `slack` rows of no sequence around."""
        had = lens.cpu().tolist()
        lens.copy_(torch.tensor([a + b for a, b in zip(had, new)], dtype=torch.int32))
        now = lens.cpu().tolist()
        batch = t.KvBatch(table.cuda(), lens, T)
        n, m = sum(new) + 2 * slack, sum(now) + slack
        plan = stack.prompt_plan(batch, n, starts(new, slack), m, starts(now, slack))
        edge = torch.zeros(slack, K)
        x = torch.cat([edge] + [r[a:b] for r, a, b in zip(rows, had, now)] + [edge]).cuda()
        stack.step(plan, x)
        torch.cuda.synchronize()
        for L, p in zip(stack.layers, plan):
            at = slack
            for b in range(B):
                q, out = p["q_rot"][at:at + new[b]], p["attn"][at:at + new[b]]
                if new[b]:
                    assert attends_right(out, q, *cached(L, table[b], now[b]), dt, True)
                at += new[b]
            assert not bool(p["attn"][:slack].any()) and not bool(p["attn"][at:].any())
        return x

    whole = stack_of(t, dt, pages)
    go(whole, total, max(total))
    turns = stack_of(t, dt, pages)
    lens.zero_()
    go(turns, [30, 0, 149], 149)
    go(turns, [40, 1, 1], 64, slack=0)
    tokens = stack_of(t, dt, pages)
    lens.zero_()
    new = ints(1, 1, 1)
    plan = tokens.plan(t.KvBatch(table.cuda(), lens, 1, new_lens=new))
    for i in range(max(total)):
        there = [int(i < n) for n in total]
        new.copy_(torch.tensor(there, dtype=torch.int32))
        lens.copy_(torch.tensor([min(i + 1, n) for n in total], dtype=torch.int32))
        x = torch.stack([r[i] if i < r.shape[0] else torch.zeros(K) for r in rows]).cuda()
        tokens.step(plan, x)
        if i in (0, 1, 64, 149):
            torch.cuda.synchronize()
            for L, p in zip(tokens.layers, plan):
                for b in range(B):
                    if there[b]:
                        assert attends_right(p["attn"][b], p["q_rot"][b], *cached(L, table[b], i + 1), dt, False)
    torch.cuda.synchronize()
    for s in (whole, turns, tokens):
        assert int(s.err.item()) == 0
        for b, n in enumerate(total):
            at = ref.slots(table[b], n, PAGE)
            for name in ("k", "v", "k_scale", "v_scale"):
                a, c = (getattr(x.layers[0]["cache"], name).cpu().transpose(1, 2)[at] for x in (whole, s))
                assert torch.equal(a, c), (name, b)


def test_drafts_behind_a_shared_prefix(t):  # noqa: F811
    """A prefix put in as a packed prompt, then steps of drafts behind it."""
    g = torch.Generator().manual_seed(5)
    P, B, T = 37, 3, 3
    pages, pre, table = ref.make_batch(g, [20] * B, T, PAGE, P)
    stack = stack_of(t, BF, pages)
    x = torch.randn(P, K, generator=g).cuda()
    stack.step(stack.prompt_plan(t.KvBatch(pre.cuda().view(1, -1), ints(P), P), P, starts([P]), P, starts([P])), x)
    lens, new = ints(0, 0, 0), ints(0, 0, 0)
    plan = stack.plan(t.KvBatch(table.cuda(), lens, T, new_lens=new, prefix_table=pre.cuda(), prefix_len=P))
    at = [0] * B
    for counts in ([3, 1, 2], [1, 3, 0], [3, 3, 3]):
        at = [a + c for a, c in zip(at, counts)]
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        stack.step(plan, torch.randn(B * T, K, generator=g).cuda())
        torch.cuda.synchronize()
        for L, p in zip(stack.layers, plan):
            pk, pv = cached(L, pre, P)
            for b, n in enumerate(counts):
                assert not bool(p["attn"][b, n:].any())
                k, v = cached(L, table[b], at[b])
                if n:
                    assert attends_right(p["attn"][b, :n], p["q_rot"][b, :n], torch.cat((pk, k)), torch.cat((pv, v)), BF, False)
    assert int(stack.err.item()) == 0
    # a prompt behind the prefix, read back whole
    n = [5, 0, 9]
    lens.copy_(torch.tensor([a + b for a, b in zip(at, n)], dtype=torch.int32))
    keys = [P + a + b for a, b in zip(at, n)]
    batch = t.KvBatch(table.cuda(), lens, 9, prefix_table=pre.cuda(), prefix_len=P)
    plan = stack.prompt_plan(batch, 14, starts(n), sum(keys), starts(keys))
    stack.step(plan, torch.randn(14, K, generator=g).cuda())
    torch.cuda.synchronize()
    for L, p in zip(stack.layers, plan):
        first = 0
        for b in range(B):
            k, v = cached(L, table[b], at[b] + n[b])
            if n[b]:
                assert attends_right(p["attn"][first:first + n[b]], p["q_rot"][first:first + n[b]],
                                     *(torch.cat(x) for x in zip(cached(L, pre, P), (k, v))), BF, True)
            first += n[b]
    assert int(stack.err.item()) == 0


def test_example_scores_prompts(t):  # noqa: F811
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("score_prompts", os.path.join(ROOT, "examples", "score_prompts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    scores, text, err = mod.talk(batch=3, turns=2, longest=90, steps=3)
    assert err == 0 and text.shape == (3, 3) and bool(((text >= 0) & (text < mod.VOCAB)).all())
    for n, (logprob, entropy, ids, best) in scores:
        assert logprob.shape[0] == sum(n) and bool((logprob <= 0).all()) and bool(logprob.isfinite().all())
        assert bool((entropy >= 0).all()) and bool((entropy <= math.log(mod.VOCAB) + 1e-3).all())
        assert bool((best[:, 1:] <= best[:, :-1]).all()) and bool((ids >= 0).all())
