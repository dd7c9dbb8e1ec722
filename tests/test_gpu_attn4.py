"""trit_attn_paged4 on the GPU against softmax attention in 64 bits over the values that the
codes stand for, row by row.

Tolerances.  A score is a sum of D exact products q' c per 64 columns, times s, plus z times
a sum of q', in fp32: off by at most e = (D + 8) 2^-24 scale sum |q_i| (15 s + |z|), taken
for the case's largest (about 2^-10), a factor of 1 +- e on a probability.  P is
rounded to fp16 and P s once more, each by up to 2^-11 of a term s c (of a term z only the
first), and to 2^-25 absolutely against a bound of s times 2^-8 to 2^-11 of it: below 2^-16
for the lengths here.  fp32 sums over at most 2^12 keys a part add 2^-12.  (A prefix that is written out has its values to 2^-22 of them and 2^-25 -- of scores, less than
the room of 8 roundings in e -- and its weights rounded once.)  So |out - exact| <= (2 2^-11 + 2 e + 2^-12) sum_j p_j (s c + |z|)_j + 2^-16 +
w |exact| where the output is 16-bit, and |lse - exact| <= e + 2^-12 + 2^-22 |exact|."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
from test_gpu_attn_paged import BF, CASES, F32, HF, UNIT, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def build_case(lens, T, new, hq, hkv, D, page, dt, prefix=0, nhd=False, seed=0, sharp=1.0):
    """A cache whose unused slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    pages, pre, table = ref.make_batch(g, lens, T, page, prefix)
    four = pr.random_cache(g, pages, hkv, page, D, nhd)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for row, n in [(pre, prefix)] + [(table[b], n) for b, n in enumerate(lens)]:
        if n:
            used[ref.slots(row, n, page)] = True
    for x in four[2:]:
        x.permute(0, 2, 1, 3, 4)[~used] = math.nan
    q = (sharp * torch.randn(len(lens), T, hq, D, generator=g)).to(dt)
    return dict(lens=lens, T=T, new=new, hq=hq, hkv=hkv, D=D, page=page, dt=dt, prefix=prefix, pre=pre, table=table,
                four=four, q=q)


def make_job(t, c, out_dt, scale=None, workspace=None, q=None):  # noqa: F811
    B = len(c["lens"])
    dn = None if c["new"] is None else torch.tensor(c["new"], dtype=torch.int32).cuda()
    batch = t.KvBatch(c["table"].cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda(), c["T"], new_lens=dn,
                      prefix_table=c["pre"].cuda(), prefix_len=c["prefix"])
    out = torch.full((B, c["T"], c["hq"], c["D"]), 7.0, dtype=out_dt, device="cuda")
    lse = torch.full((B, c["T"], c["hq"]), 7.0, device="cuda")
    return t.Attn4Job(t.Kv4Cache(*(pr.on_gpu(x) for x in c["four"])), batch, c["q"].cuda() if q is None else q, out, lse=lse,
                      scale=scale, workspace=workspace)


def check(c, out, lse, out_dt, scale=None):
    D, T, P = c["D"], c["T"], c["prefix"]
    scale = D ** -0.5 if scale is None else scale
    k, v = (pr.values(c["four"][i], c["four"][2 + i]).permute(0, 2, 1, 3) for i in (0, 1))
    z = c["four"][3].double().permute(0, 2, 1, 3, 4)[..., 1].repeat_interleave(64, -1)
    size = (v - z).abs() + z.abs()
    ks, kz = (c["four"][2].double().permute(0, 2, 1, 3, 4)[..., i] for i in (0, 1))
    most = (15 * ks + kz.abs()).nan_to_num(0).max()
    e = float(c["q"].double().abs().sum(-1).max() * most) * abs(scale) * (D + 8) * 2.0 ** -24
    assert e < 2.0 ** -8         # (or the test would say little)
    at = ref.slots(c["pre"], P, c["page"])
    pre = k[at], v[at], size[at]
    out, lse = out.double().cpu(), lse.double().cpu()
    wo = UNIT[out_dt]
    for b, n in enumerate(c["lens"]):
        at = ref.slots(c["table"][b], n, c["page"])
        keys, vals, sizes = (torch.cat((x, y[at])) for x, y in zip(pre, (k, v, size)))
        new = T if c["new"] is None else c["new"][b]
        for i in range(T):
            see = P + max(0, n - new + i + 1) if i < new else 0
            q = c["q"][b, i].double()
            want, wl = ref.attend(q, keys[:see], vals[:see], scale)
            mag, _ = ref.attend(q, keys[:see], sizes[:see], scale)
            tol = (2 * 2.0 ** -11 + 2 * e + 2.0 ** -12) * mag + 2.0 ** -16 + wo * want.abs()
            assert bool(((out[b, i] - want).abs() <= tol).all()), (b, i)
            if see == 0:
                assert bool((lse[b, i] == -math.inf).all()) and not bool(out[b, i].any())
            else:
                assert bool(((lse[b, i] - wl).abs() <= e + 2.0 ** -12 + 2.0 ** -22 * wl.abs()).all()), (b, i)


def run(t, c, out_dt, scale=None):  # noqa: F811
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, out_dt, scale)
    for _ in range(2):
        assert t.trit_attn_paged4(job, err) is job.out
    torch.cuda.synchronize()
    check(c, job.out, job.lse, out_dt, scale)
    return int(err.item()), job


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_matches_64_bits(t, case, wide):  # noqa: F811
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=len(lens) + prefix)
    err, _ = run(t, c, F32 if wide else dt)
    assert err == 0


MANY = [
    # lens, T, new, heads, key heads, D, page, type, prefix, order: all behind a prefix that is written out
    ([5, 300, 0, 70] * 10, 1, None, 20, 5, 128, 64, BF, 4101, False),
    ([60 + 7 * i for i in range(24)], 5, [i % 6 for i in range(24)], 24, 8, 64, 16, HF, 1501, True),
    ([9, 40] * 20, 4, None, 8, 1, 128, 48, HF, 2049, False),
    ([3] * 52, 5, [5, 0, 1, 3] * 13, 7, 7, 64, 5, BF, 999, False),
    ([64] * 100, 1, None, 32, 8, 128, 128, HF, 1024, True),
    ([17] * 33, 1, None, 24, 6, 64, 16, BF, 8200, False),
]


@pytest.mark.parametrize("case", MANY)
@pytest.mark.parametrize("wide", [False, True])
def test_many_rows_behind_a_prefix(t, case, wide):  # noqa: F811
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=prefix)
    rows, columns = len(lens) * T * (hq // hkv), prefix * hkv * D
    assert rows * columns >= (1e8 if rows > 128 else 3.2e8)      # (or this would be another kernel's test)
    err, job = run(t, c, F32 if wide else dt)
    assert err == 0 and job.workspace.numel() > 8 * columns


def test_written_out_prefix_captured_shared_and_beside_another(t):  # noqa: F811
    """A call that writes its prefix out and one of other sizes share a workspace in turn, captured and replayed
    with other queries; on two streams, each with a workspace, both as alone."""
    cases = [build_case([40] * 70, 1, None, 20, 5, 128, 64, BF, 2500, seed=1),
             build_case([500, 30, 0], 2, None, 8, 2, 64, 16, HF, 100, seed=2)]
    jobs = [make_job(t, c, c["dt"]) for c in cases]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for j in jobs:
        t.trit_attn_paged4(j, err)
    torch.cuda.synchronize()
    alone = [(j.out.clone(), j.lse.clone()) for j in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, j in zip(streams, jobs):
            t.trit_attn_paged4(j, err, stream=s)
    torch.cuda.synchronize()
    for j, (out, lse) in zip(jobs, alone):
        assert torch.equal(j.out, out) and torch.equal(j.lse, lse)
    ws = torch.zeros(max(j.workspace.numel() for j in jobs), dtype=torch.uint8, device="cuda")
    queries = [c["q"].cuda() for c in cases]
    shared = [make_job(t, c, c["dt"], workspace=ws, q=q) for c, q in zip(cases, queries)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j in shared + shared[:1]:
            t.trit_attn_paged4(j, err)
    graph.replay()
    torch.cuda.synchronize()
    for j, (out, lse) in zip(shared, alone):
        assert torch.equal(j.out, out) and torch.equal(j.lse, lse)
    for c, q in zip(cases, queries):
        c["q"] = c["q"].flip(0)
        q.copy_(c["q"])
    graph.replay()
    torch.cuda.synchronize()
    for c, j in zip(cases, shared):
        check(c, j.out, j.lse, c["dt"])
    assert int(err.item()) == 0


@pytest.mark.parametrize("scale", [-0.03, 0.0])
def test_many_rows_scales_and_bad_pages(t, scale):  # noqa: F811
    c = build_case([30] * 60, 1, None, 20, 5, 128, 16, BF, 3000)
    for x in c["four"][2:]:
        x.nan_to_num_(0.0)
    err, _ = run(t, c, F32, scale)
    assert err == 0
    d = dict(c, pre=c["pre"].clone())
    d["pre"][7], d["pre"][100] = -1, 10 ** 6
    flag, job = torch.zeros(1, dtype=torch.int32, device="cuda"), make_job(t, d, F32, scale)
    t.trit_attn_paged4(job, flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == t.ERR_INDEX and bool(job.out.isfinite().all())


@pytest.mark.parametrize("scale", [0.02, -0.03, 0.0])
@pytest.mark.parametrize("dt", [BF, HF])
def test_scales_of_any_sign(t, dt, scale):  # noqa: F811
    c = build_case([5, 300, 1000], 2, [2, 1, 2], 8, 2, 128, 16, dt, 70, sharp=3.0)
    err, _ = run(t, c, dt, scale)
    assert err == 0


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 40])
def test_queries_of_any_size(t, size):  # noqa: F811
    """A row's power of two brings bf16 queries of any size into fp16's range."""
    c = build_case([5, 300, 400], 1, None, 8, 2, 64, 16, BF)
    c["q"] = c["q"] * size
    err, _ = run(t, c, BF, 64 ** -0.5 / size)
    assert err == 0


def test_pairs_of_very_different_sizes(t):  # noqa: F811
    """s of V grows a millionfold along the keys, falls again, is 0 and subnormal."""
    c = build_case([2000], 1, None, 4, 1, 128, 16, HF, seed=5)
    at = ref.slots(c["table"][0], 2000, 16)
    s = c["four"][3].permute(0, 2, 1, 3, 4)
    f = torch.cat((10.0 ** torch.linspace(-4, 2, 1500), 10.0 ** torch.linspace(2, -3, 500)))
    x = s[at].float() * f[:, None, None, None]
    x[100:140] = 0.0
    x[7, :, :, 0] = 2.0 ** -24
    s[at] = x.half()
    err, _ = run(t, c, HF)
    assert err == 0


NONFINITE = [
    ([9, 40, 8], 4, [4, 2, 3], 8, 2, 64, 16, HF, 0, False),
    ([3000, 5], 8, [8, 3], 20, 5, 128, 16, BF, 0, False),
    ([150, 131], 130, [130, 77], 8, 2, 64, 16, BF, 0, False),
    ([2, 30, 16, 6], 5, [2, 5, 0, 1], 6, 3, 64, 9, BF, 333, True),
]


@pytest.mark.parametrize("case", NONFINITE)
@pytest.mark.parametrize("what", [2, 3])
def test_only_rows_that_see_a_nan_change(t, case, what):  # noqa: F811
    """The last token's key or value is NaN in its first group (one that held a NaN): its own rows are,
    and the rows of the tokens before it are as with that pair 0."""
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=3)
    x = c["four"][what].permute(0, 2, 1, 3, 4)
    bad = {}
    for b, n in enumerate(lens):
        m = T if new is None else new[b]
        if m < 2 or n < m:
            continue
        pg, sl = ref.slots(c["table"][b], n, page)
        x[pg[n - 1], sl[n - 1], :, 0] = torch.tensor([0.0, math.nan], dtype=torch.float16)
        bad[b] = m - 1
    assert bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, dt)
    t.trit_attn_paged4(job, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    out = job.out.cpu()
    for b, i in bad.items():
        n = lens[b]
        pg, sl = ref.slots(c["table"][b], n, page)
        assert bool(out[b, i].isnan().any(-1).all()) and not bool(out[b, :i].isnan().any())
        if what == 3:
            assert not bool(out[b, i, :, 64:].isnan().any())
        x[pg[n - 1], sl[n - 1], :, 0] = 0.0
    again = make_job(t, c, dt)
    t.trit_attn_paged4(again, err)
    torch.cuda.synchronize()
    check(c, again.out, again.lse, dt)
    for b in range(len(lens)):
        for i in range(T):
            if bad.get(b) != i:
                assert torch.equal(job.out[b, i], again.out[b, i]) and torch.equal(job.lse[b, i], again.lse[b, i])


def test_flags(t):  # noqa: F811
    """A page outside the cache reads as zeros, a length outside the table is clamped: flagged."""
    for lens, prefix in (([5, 9], 0), ([5, 9], 40)):
        c = build_case(lens, 1, None, 4, 1, 64, 4, BF, prefix)
        for x in c["four"][2:]:
            x.nan_to_num_(0.0)
        for what in ("page", "prefix", "len", "new"):
            if what == "prefix" and not prefix:
                continue
            d = dict(c, table=c["table"].clone(), pre=c["pre"].clone(), lens=list(lens))
            if what == "page":
                d["table"][1, 1] = 10 ** 6
            elif what == "prefix":
                d["pre"][3] = -1
            elif what == "len":
                d["lens"] = [5, 4 * c["table"].shape[1] + 1]
            else:
                d["new"] = [2, 1]
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            job = make_job(t, d, BF)
            t.trit_attn_paged4(job, err)
            torch.cuda.synchronize()
            assert int(err.item()) == t.ERR_INDEX, what
            assert bool(job.out.isfinite().all())


def test_strided_queries_shared_workspace_and_graph(t):  # noqa: F811
    """Queries as a view of a fused buffer; jobs of different sizes sharing a workspace in turn; both
    captured, replayed with other lengths."""
    a = build_case([700, 3000], 1, None, 8, 2, 64, 16, BF, 0)
    b = build_case([33, 900, 5], 2, None, 8, 1, 128, 64, HF, 100)
    fused = torch.randn(2, 1, 12, 64).to(BF)
    fused[:, :, :8] = a["q"]
    jobs = [make_job(t, a, BF, q=fused.cuda()[:, :, :8]), make_job(t, b, HF)]
    size = max(j.workspace.numel() for j in jobs)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    shared = [make_job(t, a, BF, workspace=ws, q=fused.cuda()[:, :, :8]), make_job(t, b, HF, workspace=ws)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for j, c, dt in ((jobs[0], a, BF), (jobs[1], b, HF)):
        t.trit_attn_paged4(j, err)
        check(c, j.out, j.lse, dt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j in shared:
            t.trit_attn_paged4(j, err)
    for _ in range(3):
        for j in shared:
            j.out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for j, k in zip(shared, jobs):
            assert torch.equal(j.out, k.out) and torch.equal(j.lse, k.lse)
    lens = shared[0]._keep[1].keep[1]
    lens.copy_(torch.tensor([64, 2047], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(dict(a, lens=[64, 2047]), shared[0].out, shared[0].lse, BF)
    assert int(err.item()) == 0


def test_two_streams_at_once(t):  # noqa: F811
    cases = [build_case([3000, 40], 3, [3, 1], 8, 2, 64, 16, HF, 0),
             build_case([900 - 20 * i for i in range(30)], 1, None, 8, 2, 128, 32, BF, 500)]
    jobs = [make_job(t, c, c["dt"]) for c in cases]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for j in jobs:
        t.trit_attn_paged4(j, err)
    torch.cuda.synchronize()
    alone = [(j.out.clone(), j.lse.clone()) for j in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, j in zip(streams, jobs):
            t.trit_attn_paged4(j, err, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(j.out, o) and torch.equal(j.lse, l) for j, (o, l) in zip(jobs, alone))
    assert int(err.item()) == 0


def test_offsets_past_31_bits(t):  # noqa: F811
    """A cache of more than 2^31 bytes of codes, read near its end."""
    pages, page, D = 70000, 256, 128
    g = torch.Generator().manual_seed(1)
    k, v = (torch.zeros(pages, 2, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, 2, page, 2, 2, dtype=torch.float16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    at = [pages - 1, 3, pages - 2]
    small = pr.random_cache(g, 3, 2, page, D)
    for big, part in zip((k, v, ks, vs), small):
        big[at] = part.cuda()
    q = torch.randn(1, 1, 8, D, generator=g).to(BF)
    out, lse = torch.empty(1, 1, 8, D, dtype=BF, device="cuda"), torch.empty(1, 1, 8, device="cuda")
    cache = t.Kv4Cache(k, v, ks, vs)
    batch = t.KvBatch(torch.tensor([at], dtype=torch.int32, device="cuda"), torch.tensor([600], dtype=torch.int32, device="cuda"), 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_attn_paged4(t.Attn4Job(cache, batch, q.cuda(), out, lse=lse), err)
    rows = [torch.empty(600, 2, D, dtype=BF, device="cuda") for _ in range(2)]
    t.trit_kv4_read(t.Read4Job(cache, batch, *rows, torch.tensor([0, 600], dtype=torch.int32, device="cuda")), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    c = dict(lens=[600], T=1, new=None, hq=8, hkv=2, D=D, page=page, dt=BF, prefix=0, pre=torch.zeros(0, dtype=torch.int32),
             table=torch.arange(3, dtype=torch.int32)[None], four=small, q=q)
    check(c, out, lse, BF)
    for i in (0, 1):
        want = pr.values(small[i], small[2 + i]).float().to(BF).permute(0, 2, 1, 3).reshape(-1, 2, D)[:600]
        assert torch.equal(rows[i].cpu(), want)
