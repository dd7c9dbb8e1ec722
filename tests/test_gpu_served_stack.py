"""The serving operators together, as a user runs them: ternary layers with
attention between their products (stack.ServedStack) and the drafted decode of
examples/draft_decode.py.

Each step's attention output is compared with softmax attention in 64 bits over
the history the step's own q, k and v buffers spell out (rotated and rounded to
the cache's type by the reference), with test_gpu_attn_paged's bound widened
by the queries' and keys' rounding: scores move by at most 2 * 2^-8 (one 16-bit
rounding, unit 2^-8, of each factor; the fp32 rotation may round either way) of
scale sum |q k| <= 2^5 here, so a probability by a factor of e^(2^-2)."""
import importlib.util
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def t():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_plane_select_gb300 import build
    build.build()
    import bit_plane_select_gb300 as t
    torch.cuda.set_device(0)
    return t


def test_prefix_then_ragged_steps(t):
    from bit_plane_select_gb300.stack import ServedStack
    K, F, D, HQ, HK, page, P, T = 192, 128, 64, 4, 2, 16, 37, 3
    lw = {}
    for n, (r, c) in dict(q=(HQ * D, K), k=(HK * D, K), v=(HK * D, K), o=(K, HQ * D), gate=(F, K), up=(F, K),
                          down=(K, F)).items():
        lw[n] = (torch.from_numpy(synth.ternary(synth.rng_for(9, r, c), r, c, synth.P_ZERO)), 0.5 / math.sqrt(c))
    lw["attn_gain"] = lw["mlp_gain"] = torch.ones(K)
    g = torch.Generator().manual_seed(4)
    B = 3
    pages, pre, table = ref.make_batch(g, [20] * B, T, page, P)
    ang = torch.arange(100, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    stack = ServedStack([lw, lw], D, t.Rope(cos.cuda(), sin.cuda()), pages, page)
    x = torch.randn(P, K, generator=g)
    fill = t.KvBatch(pre.cuda().view(1, -1), torch.tensor([P], dtype=torch.int32).cuda(), P)
    plan = stack.plan(fill)
    out = stack.step(plan, x.cuda())
    torch.cuda.synchronize()
    assert bool(out.isfinite().all())

    def rotated(rows, heads, pos):
        r = ref.rotate(rows.double().cpu().view(-1, heads, D).transpose(0, 1), cos[pos].double().T, sin[pos].double().T,
                       D, False)
        return r.transpose(0, 1).to(torch.bfloat16).double()
    hist = []          # per layer: prefix keys and values, then each sequence's own
    for L in plan:
        pk = rotated(L["k"], HK, torch.arange(P))
        pv = L["v"].cpu().to(torch.bfloat16).double().view(P, HK, D)
        hist.append([(pk, pv)] + [(pk[:0], pv[:0]) for _ in range(B)])
        check(L["attn"][0], rotated(L["q"], HQ, torch.arange(P)), [(pk[:i + 1], pv[:i + 1]) for i in range(P)])

    lens = torch.zeros(B, dtype=torch.int32).cuda()
    new = torch.zeros(B, dtype=torch.int32).cuda()
    who = t.KvBatch(table.cuda(), lens, T, new_lens=new, prefix_table=pre.cuda(), prefix_len=P)
    plan = stack.plan(who)
    at = [0] * B
    for counts in ([3, 1, 2], [1, 3, 0], [2, 2, 3]):
        at = [a + c for a, c in zip(at, counts)]
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        stack.step(plan, torch.randn(B * T, K, generator=g).cuda())
        torch.cuda.synchronize()
        for L, H in zip(plan, hist):
            for b, n in enumerate(counts):
                if n == 0:
                    assert not bool(L["attn"][b].any())
                    continue
                pos = P + at[b] - n + torch.arange(n)
                rows = slice(b * T, b * T + n)
                k, v = H[1 + b]
                k = torch.cat((k, rotated(L["k"][rows], HK, pos)))
                v = torch.cat((v, L["v"][rows].cpu().to(torch.bfloat16).double().view(n, HK, D)))
                H[1 + b] = (k, v)
                seen = [(torch.cat((H[0][0], k[:at[b] - n + i + 1])), torch.cat((H[0][1], v[:at[b] - n + i + 1])))
                        for i in range(n)]
                check(L["attn"][b], rotated(L["q"][rows], HQ, pos), seen)
    assert int(stack.err.item()) == 0


def check(got, q, seen):
    D = got.shape[-1]
    for i, (k, v) in enumerate(seen):
        room = float((q[i][:, None].abs() * k.abs().repeat_interleave(q.shape[1] // k.shape[1], 1).transpose(0, 1)).sum(-1).max())
        assert room * D ** -0.5 <= 2 ** 5
        want, _ = ref.attend(q[i], k, v, D ** -0.5)
        mag, _ = ref.attend(q[i], k, v.abs(), D ** -0.5)
        tol = (math.exp(2.0 ** -2) - 1 + 2.0 ** -7) * mag + 2.0 ** -20
        assert bool(((got[i].double().cpu() - want).abs() <= tol).all())


def example():
    spec = importlib.util.spec_from_file_location("draft_decode", os.path.join(ROOT, "examples", "draft_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_drafted_decode_runs_and_repeats(t):
    m = example()
    a, err = m.decode(batch=5, prompt=130, steps=4, drafts=3)
    b, _ = m.decode(batch=5, prompt=130, steps=4, drafts=3)
    assert err == 0
    for (x, k), (y, j) in zip(a, b):
        assert torch.equal(x, y) and torch.equal(k, j)      # nothing depends on an order of arrival
        for row, n in zip(x.tolist(), k.tolist()):
            assert 0 <= n <= 3 and all(0 <= v < m.VOCAB for v in row[:n + 1]) and all(v == -1 for v in row[n + 1:])
    with pytest.raises(ValueError):
        t.VerifyJob(torch.zeros(2, 3, 8).cuda(), torch.zeros(2, 3, 8).cuda(), *[None] * 5)


def test_served_stack_rejects_shapes_that_do_not_chain(t):
    from bit_plane_select_gb300.stack import ServedStack
    z = lambda n, k: (torch.zeros((n, k), dtype=torch.int8), 1.0)  # noqa: E731
    bad = {"q": z(128, 64), "k": z(64, 64), "v": z(64, 64), "o": z(64, 64), "gate": z(96, 64), "up": z(96, 64),
           "down": z(64, 96), "attn_gain": torch.ones(64), "mlp_gain": torch.ones(64)}
    with pytest.raises(ValueError):
        ServedStack([bad], 64, t.Rope(), 4, 16)
