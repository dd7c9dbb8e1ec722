"""trit_attn_prompt on the GPU against causal softmax attention in 64 bits.

Tolerances as test_gpu_attn_paged derives them: scores to 2^-11 (the inputs keep scale sum
|q_i k_i| below 2^6), P rounded to the 16-bit type (unit roundoff w), fp32 sums over at most
2^12 keys 2^-12:
|out - exact| <= (w + 2 * 2^-11 + 2^-12) sum_j p_j |v_j| + 2^-25 (+ w |exact| where out is 16-bit),
|lse - exact| <= 2^-11 + 2^-12 + 2^-22 |exact|."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
from test_gpu_attn_paged import BF, F32, HF, UNIT, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def build(nq, nk, hq, h, D, dt, seed=0, slack=2, sharp=1.0):
    """Packed CPU tensors with `slack` rows in front of, and behind, the sequences."""
    g = torch.Generator().manual_seed(seed)
    qs, ks = (torch.tensor([slack] + n, dtype=torch.int64).cumsum(0) for n in (nq, nk))
    q = (sharp * torch.randn(int(qs[-1]) + slack, hq, D, generator=g)).to(dt)
    k, v = (torch.randn(int(ks[-1]) + slack, h, D, generator=g).to(dt) for _ in range(2))
    for x, bad in ((k, NAN), (v, INF)):       # what lies in no sequence is poison
        x[:slack], x[int(ks[-1]):] = bad, bad
    return dict(nq=nq, nk=nk, q=q, k=k, v=v, qs=qs, ks=ks, dt=dt, D=D, hq=hq, h=h)


def make(t, c, out_dt, scale=None, starts_of_keys=True):  # noqa: F811
    out = torch.full(c["q"].shape, 7.0, dtype=out_dt, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    return t.PromptJob(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), out, c["qs"].to(torch.int32).cuda(),
                       c["ks"].to(torch.int32).cuda() if starts_of_keys else None, lse=lse, scale=scale)


def check(c, job, scale=None):
    D, dt = c["D"], c["dt"]
    scale = D ** -0.5 if scale is None else scale
    out, lse = job.out.double().cpu(), job.lse.double().cpu()
    w, wo = UNIT[dt], UNIT[job.out.dtype]
    used = torch.zeros(out.shape[0], dtype=torch.bool)
    for b, (n, m) in enumerate(zip(c["nq"], c["nk"])):
        rows = slice(int(c["qs"][b]), int(c["qs"][b]) + n)
        used[rows] = True
        keys = slice(int(c["ks"][b]), int(c["ks"][b]) + m)
        want, wl, mag = pr.causal(c["q"][rows].double(), c["k"][keys].double(), c["v"][keys].double(), scale)
        tol = (w + 2.0 ** -10 + 2.0 ** -12) * mag + wo * want.abs() + 2.0 ** -25
        assert bool(((out[rows] - want).abs() <= tol).all()), b
        none = wl == -INF
        assert bool((lse[rows][none] == -INF).all())
        assert bool(((lse[rows] - wl).abs() <= 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -22 * wl.abs())[~none].all()), b
    assert bool((out[~used] == 7.0).all()) and bool((lse[~used] == 7.0).all())


def run(t, c, out_dt, scale=None, **kw):  # noqa: F811
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make(t, c, out_dt, scale, **kw)
    for _ in range(2):
        assert t.trit_attn_prompt(job, err) is job.out
    torch.cuda.synchronize()
    check(c, job, scale)
    return int(err.item()), job


CASES = [
    # queries, keys (None: the same), Hq, heads, D, type
    ([1], None, 20, 5, 128, BF),
    ([700], None, 20, 5, 128, BF),
    ([64, 65, 63, 1, 129, 0, 32], None, 8, 2, 128, HF),
    ([33, 300, 5], None, 4, 4, 64, BF),
    ([255, 256, 257], None, 8, 1, 64, HF),
    ([130, 7], None, 7, 7, 128, BF),
    ([90, 41], None, 21, 3, 64, BF),                # seven heads to a key head: two rows of a tile idle
    ([50, 3], None, 10, 2, 128, HF),                # five
    ([20, 1], None, 130, 1, 64, BF),                # more heads to a key head than rows of a tile
    ([9, 2], None, 300, 2, 64, HF),
    ([1, 5, 0, 300], [1000, 5, 40, 777], 20, 5, 128, BF),          # behind earlier keys
    ([40, 3, 129], [41, 515, 130], 24, 8, 64, HF),
    ([10, 200, 7, 5], [4, 130, 0, 5], 8, 2, 128, BF),              # fewer keys than queries
    ([1] * 90, None, 4, 1, 64, BF),
    ([(i * 37) % 200 for i in range(75)], None, 4, 2, 64, HF),
    ([1500], None, 6, 2, 128, HF),
    # more tiles than SMs: two CTAs an SM
    ([1500], None, 20, 5, 128, BF),
    ([700, 1, 0, 333], [1100, 900, 7, 333], 24, 8, 64, HF),        # a few an SM: by length
    ([300 + i for i in range(33)], None, 8, 4, 64, BF),            # many sequences: in their order
    ([(i * 53) % 260 for i in range(70)], [(i * 53) % 260 + i for i in range(70)], 20, 5, 128, HF),
    ([3, 200], [2, 90], 600, 100, 64, BF),                         # and fewer keys than queries
    ([1030, 517], [2050, 517], 4, 1, 64, BF),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_matches_64_bits(t, case, wide):  # noqa: F811
    nq, nk, hq, h, D, dt = case
    c = build(nq, nk or nq, hq, h, D, dt, seed=len(nq) + D)
    err, _ = run(t, c, F32 if wide else dt, starts_of_keys=nk is not None)
    assert err == 0


@pytest.mark.parametrize("dt", [BF, HF])
def test_rising_scores_and_any_scale(t, dt):  # noqa: F811
    """Sharp scores whose maxima grow from block to block."""
    c = build([900, 130], [1400, 130], 8, 2, 64, dt, sharp=6.0)
    c["k"][2:1402] = (c["k"][2:1402].float() * torch.linspace(0.1, 1.0, 1400)[:, None, None]).to(dt)
    for scale in (None, 0.01):
        err, _ = run(t, c, dt, scale)
        assert err == 0


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("hq,h,D,dt", [(8, 2, 64, HF), (20, 5, 128, BF), (3, 3, 128, BF)])
def test_only_rows_that_see_a_bad_value_change(t, hq, h, D, dt, value):  # noqa: F811
    nq, nk = [300, 40, 5], [300, 170, 5]
    c = build(nq, nk, hq, h, D, dt, seed=9)
    at = [(0, 131, 5), (0, 140, 7), (0, 299, 1), (1, 150, 9), (2, 2, 4), (2, 4, 4)]
    for b, j, col in at:
        c["v"][int(c["ks"][b]) + j, :, col] = value
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make(t, c, dt)
    t.trit_attn_prompt(job, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    out = job.out.double().cpu()
    w = UNIT[dt]
    for b, (n, m) in enumerate(zip(nq, nk)):
        rows = slice(int(c["qs"][b]), int(c["qs"][b]) + n)
        keys = slice(int(c["ks"][b]), int(c["ks"][b]) + m)
        want, _, mag = pr.causal(c["q"][rows].double(), c["k"][keys].double(), c["v"][keys].double().nan_to_num(0, 0, 0), D ** -0.5)
        tol = (w + 2.0 ** -10 + 2.0 ** -12) * mag + w * want.abs() + 2.0 ** -25
        for i in range(n):
            row = out[rows][i]
            cols = sorted({col for bb, j, col in at if bb == b and j < m - n + i + 1})
            keep = torch.ones(D, dtype=torch.bool)
            keep[cols] = False
            assert bool(((row - want[i]).abs() <= tol[i])[:, keep].all()), (b, i)
            if cols:
                assert bool(row[:, cols].isnan().all()) if value != value else bool((row[:, cols] == value).all()), (b, i)


@pytest.mark.parametrize("value", [INF, NAN])
def test_only_rows_that_see_a_bad_key_change(t, value):  # noqa: F811
    c = build([300, 40], [300, 170], 8, 2, 64, BF, seed=9)
    at = [(0, 131), (0, 299), (1, 150)]
    first = {0: 131, 1: 150}
    for b, j in at:
        c["k"][int(c["ks"][b]) + j, :, 3] = value
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make(t, c, BF)
    t.trit_attn_prompt(job, err)
    torch.cuda.synchronize()
    out = job.out.double().cpu()
    clean = c["k"].double().nan_to_num(0, 0, 0)
    for b, (n, m) in enumerate(zip(c["nq"], c["nk"])):
        rows, keys = slice(int(c["qs"][b]), int(c["qs"][b]) + n), slice(int(c["ks"][b]), int(c["ks"][b]) + m)
        want, _, mag = pr.causal(c["q"][rows].double(), clean[keys], c["v"][keys].double(), 64 ** -0.5)
        free = first[b] - (m - n)           # queries before it do not see the first bad key
        tol = (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12) * mag + 2.0 ** -8 * want.abs() + 2.0 ** -25
        assert bool(((out[rows] - want).abs() <= tol)[:free].all())
        if value != value:
            assert bool(out[rows][free:].isnan().all())


def test_strided_rows(t):  # noqa: F811
    """q, k and v as views of one fused buffer."""
    c = build([200, 61], [200, 61], 8, 2, 64, BF)
    fused = torch.cat([c[x].flatten(1) for x in "qkv"], 1).cuda()
    q, k, v = (x.unflatten(1, (-1, 64)) for x in torch.split(fused, [512, 128, 128], 1))
    out = torch.full(c["q"].shape, 7.0, dtype=BF, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    job = t.PromptJob(q, k, v, out, c["qs"].to(torch.int32).cuda(), lse=lse)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_attn_prompt(job, err)
    torch.cuda.synchronize()
    check(c, job)
    assert int(err.item()) == 0


def test_bad_starts_are_flagged(t):  # noqa: F811
    """Starts that fall or leave the rows: flagged, and the good sequences are right."""
    for which, at, to in (("qs", 2, 5), ("qs", 3, 10 ** 6), ("ks", 0, -1), ("ks", 3, 2 ** 31 - 1)):
        c = build([100, 60, 33], [100, 160, 33], 8, 2, 64, HF)
        d = dict(c, qs=c["qs"].clone(), ks=c["ks"].clone())
        d[which][at] = to
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = make(t, d, HF)
        t.trit_attn_prompt(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == t.ERR_INDEX
        for b in {0: [1, 2], 2: [0], 3: [0, 1]}[at]:
            rows = slice(int(c["qs"][b]), int(c["qs"][b + 1]))
            keys = slice(int(c["ks"][b]), int(c["ks"][b + 1]))
            want, _, mag = pr.causal(c["q"][rows].double(), c["k"][keys].double(), c["v"][keys].double(), 64 ** -0.5)
            assert bool(((job.out[rows].double().cpu() - want).abs() <= 2.0 ** -8 * (mag + want.abs()) + 2.0 ** -25).all())


def test_without_keys(t):  # noqa: F811
    q = torch.randn(9, 4, 64).to(BF).cuda()
    k = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((9, 4), 7.0, device="cuda")
    starts = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1, 5, 8], [0, 0, 0])]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_attn_prompt(t.PromptJob(q, k, k, out, *starts, lse=lse), err)
    torch.cuda.synchronize()
    assert not bool(out[1:8].any()) and bool((out[[0, 8]] == 7.0).all())
    assert bool((lse[1:8] == -INF).all()) and bool((lse[[0, 8]] == 7.0).all()) and int(err.item()) == 0


def test_replayed_on_other_starts_and_two_streams(t):  # noqa: F811
    a, b = build([300, 100, 40], [300, 400, 40], 20, 5, 128, BF), build([600, 1], [600, 900], 8, 8, 64, HF)
    jobs = [make(t, a, BF), make(t, b, HF)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for j, c in zip(jobs, (a, b)):
        t.trit_attn_prompt(j, err)
        torch.cuda.synchronize()
        check(c, j)
    alone = [j.out.clone() for j in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, j in zip(streams, jobs):
            t.trit_attn_prompt(j, err, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(j.out, o) for j, o in zip(jobs, alone))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j in jobs:
            t.trit_attn_prompt(j, err)
    d = dict(a, nq=[2, 397, 41], nk=[3, 600, 137], qs=torch.tensor([2, 4, 401, 442]), ks=torch.tensor([2, 5, 605, 742]))
    jobs[0]._keep[4].copy_(d["qs"])
    jobs[0]._keep[5].copy_(d["ks"])
    for j in jobs:
        j.out.fill_(7.0)
        j.lse.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check(d, jobs[0])
    assert torch.equal(jobs[1].out[2:603], alone[1][2:603]) and int(err.item()) == 0
