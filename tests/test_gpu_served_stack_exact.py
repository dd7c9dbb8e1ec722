"""ServedStack's attention, operand by operand: each step's rotated queries and appended
cache slots against the rotation of the step's own fp32 products (test_gpu_kv_append's
bound, one rounding), then the attention's output against 64-bit softmax attention over the
queries and the cache's contents as they lie on the device (test_gpu_attn_paged's
bound for an fp32 output).  Scores spread over several units, and the same checks are
shown to fail for a key left out, a key too many, the own keys lost, a shifted position
and other queries."""
import math

import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
import synth  # noqa: E402
from test_gpu_attn_paged import BF, HF, UNIT, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu
K, F, D, HQ, HK, P, T, B = 192, 128, 64, 4, 2, 37, 3, 3


def layer(seed):
    """Products of q and k of about 1.6, so scores of about 2.5, and v of about 0.4."""
    lw = {}
    for n, (r, c) in dict(q=(HQ * D, K), k=(HK * D, K), v=(HK * D, K), o=(K, HQ * D), gate=(F, K), up=(F, K),
                          down=(K, F)).items():
        w = torch.from_numpy(synth.ternary(synth.rng_for(seed, r, c), r, c, synth.P_ZERO))
        lw[n] = (w, (2.0 if n in "qk" else 0.5) / math.sqrt(c))
    lw["attn_gain"] = lw["mlp_gain"] = torch.ones(K)
    return lw


def rotated(rows, heads, cos, sin, pos):
    """fp32 products [n, heads * D] turned to their positions, in 64 bits."""
    x = rows.double().cpu().view(-1, heads, D)
    return torch.stack([ref.rotate(x[i], cos[p].double(), sin[p].double(), D, False) for i, p in enumerate(pos)])


def turned_right(got, want, dt):
    big = 2 * want.abs().amax(-1, keepdim=True)
    tol = UNIT[dt] * want.abs() + (D + 12) * 2.0 ** -24 * big * (1 + UNIT[dt]) + 2.0 ** -25
    return bool(((got.double().cpu() - want).abs() <= tol).all())


def attends_right(got, q, keys, vals, dt):
    room = (q[:, None].abs() * keys.abs().repeat_interleave(HQ // HK, 1).transpose(0, 1)).sum(-1).max()
    assert float(room) * D ** -0.5 < 2 ** 6
    want, _ = ref.attend(q, keys, vals, D ** -0.5)
    mag, _ = ref.attend(q, keys, vals.abs(), D ** -0.5)
    return bool(((got.double().cpu() - want).abs() <= (UNIT[dt] + 2.0 ** -10 + 2.0 ** -12) * mag + 2.0 ** -25).all())


@pytest.mark.parametrize("dt", [BF, HF])
def test_every_operand_of_a_step(t, dt):  # noqa: F811
    from bit_plane_select_gb300.stack import ServedStack
    g = torch.Generator().manual_seed(4)
    page = 16
    pages, pre, table = ref.make_batch(g, [20] * B, T, page, P)
    ang = torch.arange(100, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    stack = ServedStack([layer(9), layer(10)], D, t.Rope(cos.cuda(), sin.cuda()), pages, page, dtype=dt)

    def cached(i, row, n):
        """Keys and values [n, HK, D] of layer i that a table row names."""
        at = ref.slots(row, n, page)
        c = stack.layers[i]["cache"]
        return [x.cpu().permute(0, 2, 1, 3)[at].double() for x in (c.k, c.v)]

    fill = t.KvBatch(pre.cuda().view(1, -1), torch.tensor([P], dtype=torch.int32).cuda(), P)
    plan = stack.plan(fill)
    stack.step(plan, torch.randn(P, K, generator=g).cuda())
    torch.cuda.synchronize()
    prefix = []
    for i, L in enumerate(plan):
        k, v = cached(i, pre, P)
        assert turned_right(k, rotated(L["k"], HK, cos, sin, range(P)), dt)
        assert turned_right(v, L["v"].double().cpu().view(P, HK, D), dt)
        assert turned_right(L["q_rot"][0], rotated(L["q"], HQ, cos, sin, range(P)), dt)
        for j in range(P):
            assert attends_right(L["attn"][0, j], L["q_rot"][0, j].double().cpu(), k[:j + 1], v[:j + 1], dt), (i, j)
        prefix.append((k, v))

    lens, new = (torch.zeros(B, dtype=torch.int32).cuda() for _ in range(2))
    plan = stack.plan(t.KvBatch(table.cuda(), lens, T, new_lens=new, prefix_table=pre.cuda(), prefix_len=P))
    before = [[cached(i, table[b], 0) for b in range(B)] for i in range(2)]
    seen = dict.fromkeys(("left out", "too many", "own lost", "uniform", "other heads"), 0)
    rows = 0
    at = [0] * B
    for counts in ([3, 1, 2], [1, 3, 0], [2, 2, 3], [3, 3, 3]):
        at = [a + c for a, c in zip(at, counts)]
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        stack.step(plan, torch.randn(B * T, K, generator=g).cuda())
        torch.cuda.synchronize()
        for i, L in enumerate(plan):
            for b, n in enumerate(counts):
                k, v = cached(i, table[b], at[b])
                was = at[b] - n
                assert torch.equal(k[:was], before[i][b][0]) and torch.equal(v[:was], before[i][b][1])
                before[i][b] = (k, v)
                assert not bool(L["attn"][b, n:].any()) and not bool(L["q_rot"][b, n:].any())
                if n == 0:
                    continue
                part, pos = slice(b * T, b * T + n), [P + was + j for j in range(n)]
                assert turned_right(k[was:], rotated(L["k"][part], HK, cos, sin, pos), dt)
                assert turned_right(v[was:], L["v"][part].double().cpu().view(n, HK, D), dt)
                assert turned_right(L["q_rot"][b, :n], rotated(L["q"][part], HQ, cos, sin, pos), dt)
                assert not turned_right(L["q_rot"][b, :n], rotated(L["q"][part], HQ, cos, sin, [x + 1 for x in pos]), dt)
                assert not turned_right(k[was:], rotated(L["k"][part], HK, cos, sin, [x - 1 for x in pos]), dt)
                pk, pv = prefix[i]
                for j in range(n):
                    own = was + j + 1
                    q, got = L["q_rot"][b, j].double().cpu(), L["attn"][b, j]
                    keys, vals = torch.cat((pk, k)), torch.cat((pv, v))
                    assert attends_right(got, q, keys[:P + own], vals[:P + own], dt), (i, b, j)
                    # what must not pass: counted over all rows
                    rows += 1
                    seen["left out"] += not attends_right(got, q, keys[:P + own - 1], vals[:P + own - 1], dt)
                    more = [torch.cat((x[:P + own], x[:1])) for x in (keys, vals)]
                    seen["too many"] += not attends_right(got, q, *more, dt)
                    seen["own lost"] += not attends_right(got, q, pk, pv, dt)
                    seen["uniform"] += not attends_right(got, q * 0, keys[:P + own], vals[:P + own], dt)
                    seen["other heads"] += not attends_right(got, q.flip(0), keys[:P + own], vals[:P + own], dt)
    assert int(stack.err.item()) == 0
    assert all(n > rows // 2 for n in seen.values()), (rows, seen)
