"""trit_kv4_append and trit_kv4_read on the GPU.

The codes of a key follow from its fp32 values: without head norms every slot is
compared bit by bit with the format's definition (prompt_ref.quantised of values turned in
fp32, operation by operation).  With a norm, whose sum may be added up in any order, a stored
value is held to half a step of the exact one: |s c + z - x| <= s/2 + rounding of s and z
to fp16 (15 s 2^-11 and |z| 2^-11) + the norm's and rotation's fp32 error (D + 14)
2^-24 (|a| + |b|), as derived in test_gpu_kv_append.  Values read back are the fp32 s c + z
rounded once."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
from test_gpu_kv_append import UNIT, t, tables  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def up(x):
    return None if x is None else x.cuda()


def make(t, lens, T, new, hq, hkv, D, rot, page, dt, src, norm, pairs, prefix=0, nhd=False, packed=False, seed=0,  # noqa: F811
         plant=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages, pre, table = ref.make_batch(g, lens, T, page, prefix)
    four = pr.random_cache(g, pages, hkv, page, D, nhd)
    n = [T] * B if new is None else new
    starts = torch.tensor([3 * packed] + n, dtype=torch.int64).cumsum(0).to(torch.int32) if packed else None
    rows = int(starts[-1]) + 2 if packed else B * T
    q, k, v = ((torch.randn(rows, h, D, generator=g) * 3).to(src) for h in (hq, hkv, hkv))
    if plant:
        plant(q, k, v)
    cos, sin = tables(prefix + max(lens) + 1, rot) if rot else (None, None)
    gq, gk = (torch.rand(D, generator=g) + 0.5 for _ in range(2)) if norm else (None, None)
    cache = t.Kv4Cache(*(pr.on_gpu(x) for x in four))
    batch = t.KvBatch(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), T,
                      new_lens=None if new is None or packed else torch.tensor(new, dtype=torch.int32).cuda(),
                      prefix_table=up(pre), prefix_len=prefix)
    q_out = torch.full((rows, hq, D) if packed else (B, T, hq, D), 7.0, dtype=dt, device="cuda")
    shape = (lambda x: x.cuda()) if packed else (lambda x: x.cuda().view(B, T, -1, D))
    rope = t.Rope(up(cos), up(sin), pairs, up(gq), up(gk), 1e-5)
    job = t.Append4Job(cache, batch, rope, shape(q), shape(k), shape(v), q_out, starts=up(starts))
    return dict(job=job, cache=cache, batch=batch, four=four, lens=lens, n=n, T=T, starts=starts, q=q, k=k, v=v, cos=cos,
                sin=sin, gq=gq, gk=gk, table=table, pre=pre, prefix=prefix, page=page, D=D, rot=rot, pairs=pairs, dt=dt,
                rows=rows, packed=packed)


CASES = [
    # lens, T, new, hq, hkv, D, rot, page, type, source, norm, pairs, prefix, nhd, packed
    ([1], 1, None, 20, 5, 128, 128, 64, BF, F32, False, False, 0, False, False),
    ([9, 1, 130], 1, None, 20, 5, 128, 128, 16, BF, F32, True, False, 77, False, False),
    ([7, 40, 16, 33], 5, [5, 0, 3, 1], 8, 2, 64, 64, 16, HF, F32, False, True, 0, True, False),
    ([7, 40, 16, 33], 5, [5, 0, 3, 1], 8, 2, 64, 48, 5, BF, BF, False, False, 1001, False, False),
    ([7, 40, 16, 33], 5, [5, 0, 3, 1], 8, 2, 64, 48, 5, BF, BF, False, False, 33, True, True),
    ([300, 5, 61], 300, [300, 5, 60], 4, 4, 128, 72, 7, HF, HF, True, False, 0, False, True),
    ([300, 5, 61], 300, [300, 5, 60], 4, 4, 128, 72, 7, HF, HF, False, False, 0, False, True),
    ([12, 5], 3, None, 7, 7, 64, 24, 1, BF, F32, True, True, 3, True, False),
    ([12, 5], 3, None, 3, 1, 128, 0, 256, HF, F32, False, False, 0, False, False),
    ([40] * 70, 2, [(i * 7) % 3 for i in range(70)], 2, 1, 64, 64, 64, BF, F32, False, False, 0, False, True),
    ([65, 64], 2, [0, 0], 2, 1, 64, 64, 64, BF, F32, False, False, 0, False, False),
]


@pytest.mark.parametrize("case", CASES)
def test_append_matches_the_format(t, case):  # noqa: F811
    c = make(t, *case)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert t.trit_kv4_append(c["job"], err) is c["job"].q_out
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    D, page, dt = c["D"], c["page"], c["dt"]
    w = UNIT[dt]
    got = [x.cpu() for x in (c["cache"].k, c["cache"].v, c["cache"].k_scale, c["cache"].v_scale)]
    want = [x.clone() for x in c["four"]]
    q_out = c["job"].q_out.cpu().view(c["rows"], -1, D)
    seen = torch.zeros(c["rows"], dtype=torch.bool)
    for b, n in enumerate(c["n"]):
        first = int(c["starts"][b]) if c["packed"] else b * c["T"]
        for i in range(n):
            row, own = first + i, c["lens"][b] - n + i
            seen[row] = True
            cos, sin = (c["cos"][c["prefix"] + own], c["sin"][c["prefix"] + own]) if c["rot"] else (None, None)
            pg, sl = int(c["table"][b, own // page]), own % page
            exact = {}
            for name, gain in (("q", c["gq"]), ("k", c["gk"])):
                x = c[name][row].double()
                if gain is not None:
                    x = torch.stack([ref.normed(y, gain.double(), 1e-5) for y in x])
                exact[name] = ref.rotate(x, None if cos is None else cos.double(), None if sin is None else sin.double(),
                                         c["rot"], c["pairs"])
            big = 2 * exact["q"].abs().amax(-1, keepdim=True)
            tol = w * exact["q"].abs() + (D + 14) * 2.0 ** -24 * big * (1 + w) + 2.0 ** -25
            assert bool(((q_out[row].double() - exact["q"]).abs() <= tol).all())
            for at, x in ((0, None if c["gk"] is not None else pr.rotate32(c["k"][row].float(), cos, sin, c["rot"], c["pairs"])),
                          (1, c["v"][row].float())):
                if x is None:
                    x = exact["k"]
                    stored = pr.values(got[0][pg, :, sl], got[2][pg, :, sl])
                    s, z = (got[2][pg, :, sl, :, j].double().repeat_interleave(64, -1) for j in (0, 1))
                    big = 2 * x.abs().amax(-1, keepdim=True)
                    tol = s / 2 + 15 * s * 2.0 ** -11 + z.abs() * 2.0 ** -11 + (D + 14) * 2.0 ** -24 * big + 2.0 ** -25
                    assert bool(((stored - x).abs() <= tol).all())
                    span = x.unflatten(-1, (-1, 64))
                    span = (span.amax(-1) - span.amin(-1)) / 15
                    assert bool((got[2][pg, :, sl, :, 0].double() <= span * (1 + 2.0 ** -10) + 2.0 ** -24).all())
                    want[0][pg, :, sl], want[2][pg, :, sl] = got[0][pg, :, sl], got[2][pg, :, sl]
                    continue
                codes, scale = pr.quantised(x)
                want[at][pg, :, sl], want[2 + at][pg, :, sl] = pr.pack(codes), scale
    for a, b in zip(got, want):      # every slot, the untouched ones among them
        assert torch.equal(a, b)
    if c["packed"]:                  # rows of no sequence stay as they were
        assert bool((q_out[~seen] == 7.0).all())
    else:
        assert not bool(q_out[~seen].any())


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("slack", [0, 5])
def test_read_gives_the_values(t, case, slack):  # noqa: F811
    c = make(t, *case)
    P, page, D = c["prefix"], c["page"], c["D"]
    starts = torch.tensor([slack] + [P + n + slack * (i % 2) for i, n in enumerate(c["lens"])], dtype=torch.int64).cumsum(0)
    rows = int(starts[-1]) + slack
    out = [torch.full((rows, c["k"].shape[1], D), 7.0, dtype=c["dt"], device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_kv4_read(t.Read4Job(c["cache"], c["batch"], *out, starts.to(torch.int32).cuda()), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for at in (0, 1):
        want = torch.full((rows, c["k"].shape[1], D), 7.0, dtype=c["dt"])
        full = pr.values(c["four"][at], c["four"][2 + at]).float().to(c["dt"]).permute(0, 2, 1, 3)
        for b, n in enumerate(c["lens"]):
            s = int(starts[b])
            want[s:s + P] = full[ref.slots(c["pre"], P, page)] if P else want[s:s]
            want[s + P:s + P + n] = full[ref.slots(c["table"][b], n, page)]
        assert torch.equal(out[at].cpu(), want)


def test_unusual_values(t):  # noqa: F811
    """Constant groups, values beyond fp16, tiny spreads, infinities and NaN."""
    def plant(q, k, v):
        for x in (k, v):
            x[0] = 1.25
            x[1] = torch.linspace(-3e5, 3e5, x.shape[-1])
            x[2] = 1 + torch.arange(x.shape[-1]) * 1e-9
            x[3, :, 5] = math.inf
            x[4, :, 70] = math.nan
            x[5] = 0.0
            x[6, :, 3] = -math.inf
    c = make(t, [8], 8, None, 2, 1, 128, 0, 16, BF, F32, False, False, plant=plant)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_kv4_append(c["job"], err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pg = int(c["table"][0, 0])
    for at, x in ((0, c["k"]), (1, c["v"])):
        codes, scale = pr.quantised(x)
        got = [(c["cache"].k, c["cache"].v)[at].cpu(), (c["cache"].k_scale, c["cache"].v_scale)[at].cpu()]
        for i in range(8):
            assert torch.equal(got[0][pg, :, i], pr.pack(codes[i]))
            assert torch.equal(got[1][pg, :, i].nan_to_num(9), scale[i].nan_to_num(9))
        z = got[1][pg, :, :, :, 1]
        assert bool(z[:, 3, 0].isnan().all()) and not bool(z[:, 3, 1].isnan().any()) and bool(z[:, 4, 1].isnan().all())


def test_index_errors_are_flagged(t):  # noqa: F811
    """A page outside the cache, a token before key 0, starts that fall or pass the rows, too many
    tokens, room for fewer keys: the flag, and nothing outside is touched."""
    D, page = 64, 4
    g = torch.Generator().manual_seed(3)

    def run(lens, new, row, starts, rows, top=64, T=3):
        four = [x.cuda() for x in pr.random_cache(g, 6, 2, page, D)]
        before = [x.clone() for x in four]
        cos, sin = (x.cuda() for x in tables(top, D))
        batch = t.KvBatch(torch.tensor([row] * len(lens), dtype=torch.int32, device="cuda"),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), T,
                          new_lens=torch.tensor(new, dtype=torch.int32, device="cuda") if new else None)
        n = rows if starts else len(lens) * T
        q, k, v = (torch.randn(n, h, D, generator=g).cuda() for h in (4, 2, 2))
        out = torch.ones((n, 4, D) if starts else (len(lens), T, 4, D), dtype=BF, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        st = torch.tensor(starts, dtype=torch.int32, device="cuda") if starts else None
        if not starts:
            q, k, v = (x.view(len(lens), T, -1, D) for x in (q, k, v))
        t.trit_kv4_append(t.Append4Job(t.Kv4Cache(*four), batch, t.Rope(cos, sin), q, k, v, out, starts=st), err)
        torch.cuda.synchronize()
        wrote = (four[0] != before[0]).any(-1).any(1)
        return int(err.item()), int(wrote.sum()), out
    E = t.ERR_INDEX
    for lens, new, row, top, good in (([1], [3], [1, 2], 64, 1), ([40], [1], [1, 2], 64, 0), ([5], [1], [1, 6], 64, 0),
                                      ([5], [1], [1, -1], 64, 0), ([8], [1], [1, 2], 7, 0), ([8], [4], [1, 2], 64, 3),
                                      ([8], [-1], [1, 2], 64, 0)):
        assert run(lens, new, row, None, 0, top)[:2] == (E, good), (lens, new, row)
    assert run([3, 3], None, [1, 2], [0, 3, 2], 6)[0] == E             # the second falls
    assert run([3], None, [1, 2], [0, 9], 3)[:2] == (E, 3)             # past the rows: what is there (T of it)
    assert run([3], None, [1, 2], [-2, 1], 3)[0] == E
    err, wrote, out = run([8], None, [1, 2], [0, 5], 6, T=3)           # five tokens where three fit
    assert (err, wrote) == (E, 3) and not bool(out[3:5].any()) and bool((out[5] == 1).all())

    four = [x.cuda() for x in pr.random_cache(g, 6, 2, page, D)]
    cache = t.Kv4Cache(*four)

    def read(lens, row, starts, rows):
        batch = t.KvBatch(torch.tensor([row] * len(lens), dtype=torch.int32, device="cuda"),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), 1)
        out = [torch.full((rows, 2, D), 7.0, dtype=BF, device="cuda") for _ in range(2)]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        t.trit_kv4_read(t.Read4Job(cache, batch, *out, torch.tensor(starts, dtype=torch.int32, device="cuda")), err)
        torch.cuda.synchronize()
        return int(err.item()), [int((x == 7.0).all(-1).all(-1).sum()) for x in out], out
    assert read([5], [1, 2], [0, 5], 7)[:2] == (0, [2, 2])
    assert read([5], [1, 2], [0, 3], 7)[:2] == (E, [4, 4])
    assert read([9], [1, 2], [0, 9], 9)[:2] == (E, [1, 1])             # longer than its table
    assert read([-1], [1, 2], [0, 2], 4)[:2] == (E, [4, 4])
    err, left, out = read([5], [1, 6], [0, 5], 5)
    assert (err, left) == (E, [0, 0]) and not bool(out[0][4:].any())
    assert read([5, 2], [1, 2], [0, 5, 3], 7)[0] == E
    assert read([5], [1, 2], [0, 9], 5)[0] == E


def test_append_and_read_on_another_stream_and_replayed(t):  # noqa: F811
    c = make(t, *CASES[4])
    P = c["prefix"]
    starts = torch.tensor([0] + [P + n for n in c["lens"]], dtype=torch.int64).cumsum(0)
    out = [torch.empty(int(starts[-1]), 2, c["D"], dtype=BF, device="cuda") for _ in range(2)]
    read = t.Read4Job(c["cache"], c["batch"], *out, starts.to(torch.int32).cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    t.trit_kv4_append(c["job"], err, stream=s)
    t.trit_kv4_read(read, err, stream=s)
    s.synchronize()
    first = [x.clone() for x in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.trit_kv4_append(c["job"], err)
        t.trit_kv4_read(read, err)
    for x, y in zip((c["cache"].k, c["cache"].v), c["four"]):
        x.copy_(pr.on_gpu(y))
    for x in out:
        x.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first)) and int(err.item()) == 0
