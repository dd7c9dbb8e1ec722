"""trit_logprobs on the GPU against its definition in 64 bits.

Tolerance.  Differences x - m are one rounding of |x - m|, held to 150; e^d by a
product with log2 e and ex2.approx (2 ulp): relative error below 2^-22 + |d| 2^-23.  A thread
adds up at most V / 512 terms of each sum and the rest is a tree of 12 levels, with the
maxima's corrections (each as an e^d) at most one per addition level: relative error of l,
weighted by e^d (|d| e^d < 1 summed against l >= 1 stays below |entropy| + ln V), at most
(V / 512 + 40) 2^-23 + 60 2^-22.  ln l and the entropy's two terms carry that and a few
roundings of values up to ln V and |x - m|."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
from test_gpu_kv_append import t  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def run(t, x, tokens, n, stride=0, offset=0):  # noqa: F811
    rows, V = x.shape
    if stride or offset:
        base = torch.full((rows * (V + stride) + offset + 8,), math.nan, dtype=x.dtype, device="cuda")
        dev = base[offset:offset + rows * (V + stride)].view(rows, V + stride)[:, :V]
        dev.copy_(x)
    else:
        dev = x.cuda()
    given, entropy = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    ids = torch.full((rows, n), 77, dtype=torch.int32, device="cuda") if n else None
    best = torch.full((rows, n), 9.0, device="cuda") if n else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_logprobs(t.LogprobJob(dev, tokens.cuda(), given, entropy, ids, best), err)
    torch.cuda.synchronize()
    return [None if y is None else y.cpu() for y in (given, entropy, ids, best)], int(err.item())


def check(got, want, V):
    eps = (V / 512 + 40) * 2.0 ** -23 + 60 * 2.0 ** -22
    for a, b, room in ((got[0], want[0], 1.0), (got[1], want[1], 2 * (math.log(V) + 1)), (got[3], want[3], 1.0)):
        if a is None:
            continue
        a = a.double()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.isinf(), b.isinf()) and bool((a[a.isinf()] == b[a.isinf()]).all())
        fine = b.isfinite()
        tol = eps * room + 2.0 ** -22 * b.abs()
        assert bool(((a - b).abs()[fine] <= tol[fine]).all()), float((a - b).abs()[fine].max())
    if got[2] is not None:
        assert torch.equal(got[2], want[2])


CASES = [
    # rows, V, n, type, extra stride, offset of the first row, values
    (1, 1, 1, F32, 0, 0, "normal"),
    (3, 2, 5, F32, 0, 0, "normal"),
    (6, 32000, 5, F32, 0, 0, "normal"),
    (5, 50257, 20, BF, 0, 0, "normal"),
    (7, 50257, 64, HF, 3, 1, "normal"),
    (2, 4099, 20, F32, 0, 3, "normal"),
    (400, 1003, 8, BF, 1, 5, "normal"),
    (9, 131072, 20, BF, 0, 0, "masked"),
    (40, 70001, 20, F32, 0, 0, "masked"),
    (310, 20011, 20, HF, 0, 0, "masked"),
    (5, 32000, 20, BF, 0, 0, "equal"),
    (3, 2001, 20, F32, 0, 0, "equal"),
    (2, 131072, 20, F32, 0, 0, "strided"),
    (310, 40000, 40, BF, 0, 0, "strided"),
    (3, 30000, 20, F32, 0, 0, "rising"),
    (4, 30000, 5, F32, 0, 0, "few"),
    (4, 8192, 0, F32, 0, 0, "normal"),
    (6, 9000, 20, F32, 0, 0, "large"),
    (6, 9000, 20, F32, 0, 0, "zeros"),
]


def inputs(rows, V, dt, how, g):
    x = 2.5 * torch.randn(rows, V, generator=g)
    if how == "masked":
        x[:, torch.rand(V, generator=g) < 0.4] = -math.inf
        x[0] = -math.inf
    elif how == "equal":
        x[:] = 1.25
        x[1:, V // 2:] = 0.5
    elif how == "strided":       # the greatest of many threads' chunks, all of one thread's
        x[:, :] = -5.0 + 0.001 * torch.rand(V, generator=g)
        c = 16 // (4 if dt is F32 else 2)
        x[:, ((torch.arange(V) // c) % 512) < 24] += 9.0
    elif how == "rising":
        x = torch.linspace(-9, 9, V).repeat(rows, 1)
        x[1] = x[1].flip(0)
    elif how == "few":
        y = torch.full_like(x, -math.inf)
        for r, n in enumerate((1, 3, 5, 12)):
            at = torch.randperm(V, generator=g)[:n]
            y[r, at] = x[r, at]
        x = y
    elif how == "large":
        x = x * 40 + torch.tensor([1e4, -1e4, 0, 3e7, -3e30, 1e-30])[:, None]
    elif how == "zeros":
        x = torch.where(torch.rand(rows, V, generator=g) < 0.5, 0.0, -0.0)
    return x.to(dt)


@pytest.mark.parametrize("case", CASES)
def test_matches_the_definition(t, case):  # noqa: F811
    rows, V, n, dt, stride, offset, how = case
    g = torch.Generator().manual_seed(rows * 7 + V)
    x = inputs(rows, V, dt, how, g)
    some = x[:8] if rows > 8 else x
    tokens = torch.randint(V, (rows,), generator=g, dtype=torch.int32)
    tokens[rows // 2] = -1
    got, err = run(t, x, tokens, n, stride, offset)
    k = some.shape[0]
    want = pr.scored(some, tokens[:k], n)
    check([None if y is None else y[:k] for y in got], want, V)
    assert err == (t.ERR_EMPTY if how == "masked" else 0)
    if rows > k:                 # the other rows against a row-wise formula
        y = x[k:].double()
        lse = torch.logsumexp(y, 1)
        w = torch.where(tokens[k:] < 0, 0.0, y.gather(1, tokens[k:].long().clamp(min=0)[:, None])[:, 0] - lse)
        fine = w.isfinite()
        assert bool(((got[0][k:].double() - w).abs()[fine] <= 2e-4).all()) and bool((got[0][k:][~fine] == -math.inf).all())


@pytest.mark.parametrize("dt", [F32, BF, HF])
@pytest.mark.parametrize("V,offset", [(40003, 0), (9001, 3), (130, 1)])
def test_masks_of_the_lowest_value_and_far_rows(t, dt, V, offset):  # noqa: F811
    """Rows masked by the type's lowest value, in part or whole and beside -inf; rows about the
    distance from 0 where differences are taken another way, and across it."""
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dt).min
    x = 2.5 * torch.randn(9, V, generator=g)
    x[0, : V // 2] = low
    x[1, V // 2:] = low
    x[2] = low
    x[3] = low
    x[3, torch.rand(V, generator=g) < 0.5] = -math.inf
    x[4] = low * 0.999 + x[4]
    far = 60000.0 if dt is HF else 2.0 ** 20
    x[5] += far
    x[6] -= far
    x[7] = far + torch.linspace(-40.0, 40.0, V)
    x[8, ::3] = -far
    x = x.to(dt)
    tokens = torch.randint(V, (9,), generator=g, dtype=torch.int32)
    got, err = run(t, x, tokens, 7, 5, offset)
    check(got, pr.scored(x, tokens, 7), V)
    assert err == 0


@pytest.mark.parametrize("dt", [F32, BF, HF])
def test_no_positive_logprob_and_no_negative_entropy(t, dt):  # noqa: F811
    """Rows of one great logit each, of sizes whose products with log2 e round either way."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(64, 3001, generator=g)
    x[torch.arange(64), torch.arange(64) * 40] = 30.0 + 61.0 * torch.rand(64, generator=g)
    x = x.to(dt)
    tokens = (torch.arange(64) * 40).int()
    got, err = run(t, x, tokens, 2)
    check(got, pr.scored(x, tokens, 2), 3001)
    assert err == 0 and bool((got[0] <= 0).all()) and bool((got[1] >= 0).all()) and bool((got[3] <= 0).all())


def test_rows_that_are_not_numbers(t):  # noqa: F811
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 40000, generator=g)
    x[0, 17] = math.nan
    x[1, 39999] = math.inf
    x[2] = -math.inf
    x[3, 20000] = math.nan
    tokens = torch.tensor([3, 5, 7, -1, 40000, -2], dtype=torch.int32)
    got, err = run(t, x, tokens, 4)
    check(got, pr.scored(x, tokens, 4), 40000)
    assert err == t.ERR_EMPTY | t.ERR_INDEX


def test_parts_of_the_answer(t):  # noqa: F811
    """Any of the outputs may be left out; the others are the same."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 6000, generator=g).cuda()
    tokens = torch.arange(5, dtype=torch.int32, device="cuda")
    a, b, c, d = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, 3, dtype=torch.int32, device="cuda"), \
        torch.empty(5, 3, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_logprobs(t.LogprobJob(x, tokens, a, b, c, d), err)
    for parts in ((tokens, 0, None, None, None), (None, None, 0, None, None), (None, None, None, 0, 0)):
        new = [None if p is None else p if p is tokens else torch.empty_like(o) for p, o in zip(parts, (tokens, a, b, c, d))]
        t.trit_logprobs(t.LogprobJob(x, *new), err)
        assert all(n is None or torch.equal(n, o) for n, o in zip(new, (tokens, a, b, c, d)))
    assert int(err.item()) == 0


def test_replayed_and_on_two_streams(t):  # noqa: F811
    g = torch.Generator().manual_seed(4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs = []
    for rows, V, n in ((6, 32000, 5), (500, 9001, 20)):
        x = torch.randn(rows, V, generator=g).cuda()
        out = [torch.empty(rows, device="cuda") for _ in range(2)] + [torch.empty(rows, n, dtype=torch.int32, device="cuda"),
                                                                     torch.empty(rows, n, device="cuda")]
        jobs.append((t.LogprobJob(x, torch.zeros(rows, dtype=torch.int32, device="cuda"), *out), out, x))
    for j, _, _ in jobs:
        t.trit_logprobs(j, err)
    torch.cuda.synchronize()
    alone = [[y.clone() for y in out] for _, out, _ in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (j, _, _) in zip(streams, jobs):
            t.trit_logprobs(j, err, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, (_, out, _) in zip(alone, jobs) for a, b in zip(w, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j, _, _ in jobs:
            t.trit_logprobs(j, err)
    for _, out, x in jobs:
        x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    for (_, out, x), w in zip(jobs, alone):
        assert torch.equal(out[2], w[2])           # the order is the same
        lse = torch.logsumexp(x.double(), 1)
        assert bool(((x.double()[:, 0] - lse - out[0].double()).abs() < 1e-4).all())
    assert int(err.item()) == 0
