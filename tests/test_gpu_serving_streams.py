"""The serving operators in a captured graph and on two streams at the same time."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_attn_paged as attn  # noqa: E402
import test_gpu_draft_verify as verify  # noqa: E402
from test_gpu_attn_paged import BF, HF, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,prefix", [(2, 0), (3, 70), (40, 700)])
def test_a_captured_step_follows_its_lengths(t, B, prefix):  # noqa: F811
    """Append, attend and verify captured once and replayed for several steps, tables and lengths
    updated in place between them: the same as calls."""
    g = torch.Generator().manual_seed(B)
    T, hq, hkv, D, page, V = 2, 8, 2, 64, 16, 130
    c = attn.build_case([60 + b % 5 for b in range(B)], T, None, hq, hkv, D, page, BF, prefix, poison=False)
    dev = {n: c[n].cuda() for n in ("k", "v", "table")}
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    batch = t.KvBatch(dev["table"], lens, T, prefix_table=c["pre"].cuda(), prefix_len=prefix)
    q, k, v = (torch.empty(B, T, h, D, device="cuda") for h in (hq, hkv, hkv))
    q_rot, out = (torch.empty(B, T, hq, D, dtype=d, device="cuda") for d in (BF, torch.float32))
    pos = torch.arange(prefix + 80)[:, None] * 0.3 ** torch.arange(D // 2)
    cache = t.KvCache(dev["k"], dev["v"])
    p, r, draft, u, race = (x.cuda() for x in verify.inputs(B, T, V, torch.float32, 3))
    tokens, kept = torch.empty(B, T + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    jobs = [t.AppendJob(cache, batch, t.Rope(pos.cos().cuda(), pos.sin().cuda()), q, k, v, q_rot),
            t.AttnJob(cache, batch, q_rot, out), t.VerifyJob(p, r, draft, u, race, tokens, kept)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        for f, j in zip((t.trit_kv_append, t.trit_attn_paged, t.trit_draft_verify), jobs):
            f(j, err)
    start = [x.clone() for x in (dev["k"], dev["v"])]
    inputs = [([5 * i + b % 3 + T for b in range(B)], [torch.randn(x.shape, generator=g) for x in (q, k, v)],
               torch.rand(B, T, generator=g)) for i in range(4)]

    def run(go):
        dev["k"].copy_(start[0])
        dev["v"].copy_(start[1])
        made = []
        for n, xs, uu in inputs:
            lens.copy_(torch.tensor(n, dtype=torch.int32))
            for x, y in zip((q, k, v), xs):
                x.copy_(y)
            u.copy_(uu)
            go()
            made.append([x.clone() for x in (q_rot, out, tokens, kept, dev["k"], dev["v"])])
        torch.cuda.synchronize()
        return made
    called = run(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    replayed = run(graph.replay)
    for a, b in zip(called, replayed):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert int(err.item()) == 0 and bool(called[-1][1].isfinite().all())


def test_two_streams_at_once(t):  # noqa: F811
    """Jobs with workspaces of their own, on two streams: each as it is alone."""
    cases = [([900 - 20 * i for i in range(40)], 1, None, 32, 16, 128, 32, BF, 2111, True),
             ([3000, 40], 3, [3, 1], 8, 2, 64, 16, HF, 0, False),
             ([700 + i for i in range(34)], 3, [1 + i % 3 for i in range(34)], 8, 1, 128, 128, HF, 1111, False),
             ([150, 131], 130, [130, 77], 8, 2, 64, 16, BF, 0, False)]
    jobs = []
    for lens, T, new, hq, hkv, D, page, dt, prefix, nhd in cases:
        jobs.append(attn.make_job(t, attn.build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=3), dt))
    x = [a.cuda() for a in verify.inputs(24, 5, 50257, torch.float32, 5)]
    tokens, kept = torch.empty(24, 6, dtype=torch.int32, device="cuda"), torch.empty(24, dtype=torch.int32, device="cuda")
    check = t.VerifyJob(*x, tokens, kept)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    alone = []
    for j in jobs:
        t.trit_attn_paged(j, err)
        torch.cuda.synchronize()
        alone.append((j.out.clone(), j.lse.clone()))
        j.out.fill_(7.0)
    t.trit_draft_verify(check, err)
    torch.cuda.synchronize()
    drawn = tokens.clone(), kept.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in (0, 2):
            for s in (0, 1):
                t.trit_attn_paged(jobs[i + s], err, stream=streams[s])
                if s == 1:
                    t.trit_draft_verify(check, err, stream=streams[s])
    torch.cuda.synchronize()
    for j, (out, lse) in zip(jobs, alone):
        assert torch.equal(j.out, out) and torch.equal(j.lse, lse)
    assert torch.equal(tokens, drawn[0]) and torch.equal(kept, drawn[1])
    assert int(err.item()) == 0
