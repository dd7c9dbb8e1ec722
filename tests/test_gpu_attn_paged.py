"""trit_attn_paged on the GPU against softmax attention in 64 bits, row by row.

Tolerances.  Scores are sums of D exact 16-bit products in fp32 (relative
D 2^-24 of sum |q_i k_i| at worst; the inputs keep scale sum |q_i k_i| below
2^6, so a score is off by less than 2^-11 at D = 128 and 2^-12 at D = 64: a
factor of 1 +- 2^-11 on a probability), 2^x to 2^-22; P is rounded to the
cache's type for the second product, unit roundoff w (2^-8 bf16, 2^-11 fp16), and
fp32 sums over at most 2^12 keys add 2^-12.  So |out - exact| <= (w + 2 * 2^-11
+ 2^-12) sum_j p_j |v_j| + (w |exact| + 2^-25 where the output is 16-bit), and
|lse - exact| <= 2^-11 + 2^-12 + 2^-22 |exact|."""
import math

import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 0.0}


@pytest.fixture(scope="module")
def t():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_plane_select_gb300 import build
    build.build()
    import bit_plane_select_gb300 as t
    torch.cuda.set_device(0)
    return t


def build_case(lens, T, new, hq, hkv, D, page, dt, prefix=0, nhd=False, seed=0, poison=True):
    """A cache whose unused slots hold NaN and infinity."""
    g = torch.Generator().manual_seed(seed)
    pages, pre, table = ref.make_batch(g, lens, T, page, prefix)
    k, v = (torch.randn(pages, hkv, page, D, generator=g).to(dt) for _ in range(2))
    if poison:
        used = torch.zeros(pages, page, dtype=torch.bool)
        for row, n in [(pre, prefix)] + [(table[b], n) for b, n in enumerate(lens)]:
            if n:
                used[ref.slots(row, n, page)] = True
        for x, bad in ((k, float("nan")), (v, float("inf"))):
            x.permute(0, 2, 1, 3)[~used] = bad
    q = torch.randn(len(lens), T, hq, D, generator=g).to(dt)
    return dict(lens=lens, T=T, new=new, hq=hq, hkv=hkv, D=D, page=page, dt=dt, prefix=prefix, pre=pre,
                table=table, k=k, v=v, q=q, nhd=nhd)


def make_job(t, c, out_dt, q=None, lse=True, scale=None):
    def up(x):
        return None if x is None else x.cuda()
    k, v = c["k"].cuda(), c["v"].cuda()
    if c["nhd"]:
        k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
    B = len(c["lens"])
    dl = torch.tensor(c["lens"], dtype=torch.int32).cuda()
    dn = None if c["new"] is None else torch.tensor(c["new"], dtype=torch.int32).cuda()
    batch = t.KvBatch(c["table"].cuda(), dl, c["T"], new_lens=dn, prefix_table=up(c["pre"]),
                      prefix_len=c["prefix"])
    out = torch.full((B, c["T"], c["hq"], c["D"]), 7.0, dtype=out_dt, device="cuda")
    L = torch.full((B, c["T"], c["hq"]), 7.0, device="cuda") if lse else None
    return t.AttnJob(t.KvCache(k, v), batch, c["q"].cuda() if q is None else q, out, lse=L, scale=scale)


def check(c, out, lse, scale=None):
    D, T, P = c["D"], c["T"], c["prefix"]
    scale = D ** -0.5 if scale is None else scale
    k, v = (x.permute(0, 2, 1, 3).double() for x in (c["k"], c["v"]))
    at = ref.slots(c["pre"], P, c["page"])
    pk, pv = k[at], v[at]
    out, w = out.double().cpu(), UNIT[c["dt"]]
    wo = UNIT[out_dtype(c)]
    for b, n in enumerate(c["lens"]):
        at = ref.slots(c["table"][b], n, c["page"])
        keys, vals = torch.cat((pk, k[at])), torch.cat((pv, v[at]))
        new = T if c["new"] is None else c["new"][b]
        for i in range(T):
            see = P + max(0, n - new + i + 1) if i < new else 0
            want, wl = ref.attend(c["q"][b, i].double(), keys[:see], vals[:see], scale)
            mag, _ = ref.attend(c["q"][b, i].double(), keys[:see], vals[:see].abs(), scale)
            tol = (w + 2.0 ** -10 + 2.0 ** -12) * mag + wo * want.abs() + 2.0 ** -25
            assert bool(((out[b, i] - want).abs() <= tol).all()), (b, i)
            if lse is not None:
                got = lse[b, i].double().cpu()
                if see == 0:
                    assert bool((got == -math.inf).all())
                else:
                    assert bool(((got - wl).abs() <= 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -22 * wl.abs()).all()), (b, i)


def out_dtype(c):
    return c.get("out_dt", c["dt"])


def run(t, c, out_dt, twice=True, scale=None):
    c["out_dt"] = out_dt
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, out_dt, scale=scale)
    for _ in range(2 if twice else 1):
        assert t.trit_attn_paged(job, err) is job.out
    torch.cuda.synchronize()
    check(c, job.out, job.lse, scale)
    return int(err.item()), job


CASES = [
    # lens, T, new, hq, hkv, D, page, cache type, prefix, nhd
    ([1], 1, None, 20, 5, 128, 64, BF, 0, False),
    ([0], 1, [0], 20, 5, 128, 64, BF, 0, False),
    ([0, 3], 1, [0, 1], 8, 2, 64, 16, HF, 0, False),
    ([700], 1, None, 20, 5, 128, 64, BF, 0, True),
    ([64, 65, 63, 1, 129], 1, None, 8, 2, 128, 16, HF, 0, False),
    ([33, 900, 5], 1, None, 4, 4, 64, 32, BF, 0, False),
    ([33, 900, 5], 1, None, 8, 1, 128, 7, BF, 0, False),       # pages that end inside a tile
    ([33, 90, 5], 2, [2, 0, 1], 8, 1, 64, 1, HF, 0, True),
    ([9, 40, 8], 8, [8, 3, 0], 20, 5, 128, 16, BF, 0, False),   # 32 rows
    ([40, 9], 9, None, 5, 1, 64, 24, HF, 0, False),             # 45 rows: two row tiles
    ([3000], 1, None, 8, 2, 128, 64, HF, 0, False),             # one item over many CTAs
    ([150, 131], 130, [130, 77], 8, 2, 64, 16, BF, 0, False),   # a chunk of prompt: many row tiles
    ([40, 33], 33, [33, 20], 4, 4, 128, 8, HF, 5, True),
    ([5, 3], 1, None, 20, 5, 128, 64, BF, 130, False),          # with a prefix
    ([5, 0, 77], 1, [1, 0, 1], 20, 5, 128, 64, BF, 1, False),
    ([0, 0], 1, [1, 1], 8, 2, 64, 16, HF, 500, False),          # nothing of their own
    ([2, 30, 16, 1], 5, [2, 5, 0, 1], 20, 5, 128, 16, BF, 1005, False),
    ([2, 30, 16, 1], 5, [2, 5, 0, 1], 6, 3, 64, 9, BF, 333, True),
    ([17] * 40, 1, None, 20, 5, 128, 32, BF, 700, False),       # 160 rows share the prefix
    ([1 + 3 * i for i in range(70)], 1, None, 8, 4, 64, 64, HF, 900, False),
    ([20 + i for i in range(33)], 3, [1 + i % 3 for i in range(33)], 8, 1, 128, 128, HF, 1111, False),
    ([1] * 300, 1, None, 4, 1, 64, 16, BF, 64, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_matches_64_bits(t, case, wide):
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=len(lens) + prefix)
    err, _ = run(t, c, F32 if wide else dt)
    assert err == 0


LONG = [
    # several blocks of 128 keys to a part: one row tile on two streams, two tiles, odd tiles
    ([3] * 40, 1, None, 32, 32, 64, 16, BF, 4000, False),
    ([5] * 34, 4, [1 + i % 4 for i in range(34)], 20, 20, 64, 64, HF, 3969, True),
    ([5] * 34, 2, None, 20, 20, 128, 256, BF, 2100, False),
    ([9] * 66, 1, None, 40, 10, 128, 32, HF, 1793, False),
    ([1] * 33, 1, None, 40, 40, 128, 16, BF, 2048, True),
]


@pytest.mark.parametrize("case", LONG)
@pytest.mark.parametrize("sharp", [1, 6, -6])
def test_long_prefix_many_rows(t, case, sharp):
    """Sharp scores make the maxima grow from block to block; a negative scale too."""
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=prefix)
    if abs(sharp) > 1:
        c["q"] *= abs(sharp)
        ramp = torch.linspace(0.1, 1.0, prefix)[:, None, None]
        at = ref.slots(c["pre"], prefix, page)
        kk = c["k"].permute(0, 2, 1, 3)
        kk[at] = (kk[at].float() * ramp).to(dt)
    err, _ = run(t, c, dt, scale=math.copysign(D ** -0.5, sharp))
    assert err == 0


@pytest.mark.parametrize("case", [
    ([500 + i for i in range(34)], 4, [1 + i % 4 for i in range(34)], 20, 20, 64, 64, HF, 3969, False),
    ([900 - 20 * i for i in range(40)], 1, None, 32, 16, 128, 32, BF, 2111, True),
    ([0, 2500] * 20, 1, [0, 1] * 20, 24, 12, 128, 16, HF, 1500, False),
    ([5] * 39 + [60000], 1, None, 8, 8, 64, 64, BF, 1000, False),      # a table far wider than most lengths
])
def test_much_own_work_beside_a_prefix(t, case):
    """The prefix cut into fewer parts and the own keys' chunks taken in turn; twice, so that what a
    call leaves for the next is seen."""
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=prefix)
    err, job = run(t, c, dt)
    assert err == 0
    first = job.out.clone()
    t.trit_attn_paged(job, torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(first, job.out)        # who takes a chunk changes no result


def test_zero_scale(t):
    """Every visible key weighs the same."""
    for lens in ([5, 9], [3] * 40):
        c = build_case(lens, 1, None, 4, 1, 64, 16, BF, 133)
        err, _ = run(t, c, BF, scale=0.0)
        assert err == 0


def test_a_bad_prefix_page_is_flagged(t):
    for lens in ([5, 9], [3] * 40):
        for bad in (-1, 9999):
            c = build_case(lens, 1, None, 4, 1, 64, 16, BF, 133, poison=False)
            c["pre"][3] = bad
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            job = make_job(t, c, BF)
            t.trit_attn_paged(job, err)
            torch.cuda.synchronize()
            assert int(err.item()) == t.ERR_INDEX and bool(job.out.isfinite().all())


def test_more_new_tokens_than_own_keys(t):
    """Tokens before own key 0 see the prefix alone (nothing, without one)."""
    for prefix in (0, 40):
        c = build_case([1, 2], 4, [4, 2], 8, 2, 64, 16, BF, prefix)
        err, _ = run(t, c, BF)
        assert err == 0


def test_strided_queries_no_lse(t):
    c = build_case([50, 7], 2, None, 8, 2, 64, 16, BF, 33)
    c["out_dt"] = BF
    room = torch.full((4, 8 * 64 + 24), float("nan"), dtype=BF, device="cuda")
    room[:, :512] = c["q"].reshape(4, 512).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, BF, q=room[:, :512], lse=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.trit_attn_paged(job, err, stream=s)
    torch.cuda.synchronize()
    check(c, job.out, None)
    assert int(err.item()) == 0


def test_bad_lengths_and_pages_are_flagged(t):
    for lens, page0 in (([-3], 1), ([1000], 1), ([20], 99), ([20], -1)):
        c = build_case([20], 1, None, 8, 2, 64, 16, BF, 0, poison=False)
        c["lens"] = lens
        c["table"][0, 0] = page0 if page0 != 1 else c["table"][0, 0]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = make_job(t, c, BF)
        t.trit_attn_paged(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == t.ERR_INDEX


def test_large_scores_and_nan(t):
    """Scores far apart do not overflow; a NaN key poisons the rows that see it and no other."""
    c = build_case([40, 41], 1, None, 4, 2, 64, 16, BF, 20, poison=False)
    c["q"] *= 8
    c["k"] *= 8
    c["out_dt"] = BF
    pg, sl = ref.slots(c["table"][1], 41, 16)
    c["k"][pg[30], 0, sl[30], 5] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, BF)
    t.trit_attn_paged(job, err)
    torch.cuda.synchronize()
    out, lse = job.out.cpu(), job.lse.cpu()
    assert bool(out[1, 0, :2].isnan().all()) and bool(lse[1, 0, :2].isnan().all())
    assert bool(out[1, 0, 2:].isfinite().all()) and bool(out[0].isfinite().all()) and bool(lse[0].isfinite().all())


def test_offsets_past_32_bits(t):
    """A cache of more than 2^32 bytes and 2^31 elements per tensor: the pages used are its last ones."""
    hkv, page, D = 8, 64, 128
    pages = (1 << 31) // (hkv * page * D) + 40
    kc, vc = (torch.empty(pages, hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    c = build_case([100, 30], 1, None, 16, 8, 128, 64, BF, 70)
    small = c["k"].shape[0]
    kc[-small:], vc[-small:] = c["k"].cuda(), c["v"].cuda()
    lift = pages - small
    c["out_dt"] = BF
    dl = torch.tensor(c["lens"], dtype=torch.int32).cuda()
    batch = t.KvBatch(c["table"].cuda() + lift, dl, 1, prefix_table=c["pre"].cuda() + lift, prefix_len=70)
    out = torch.empty(2, 1, 16, 128, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_attn_paged(t.AttnJob(t.KvCache(kc, vc), batch, c["q"].cuda(), out), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(c, out, None)


@pytest.mark.parametrize("B,page,D,prefix,own", [(40, 16, 128, 1500, 2500), (40, 64, 64, 1537, 2500),
                                                 (70, 32, 128, 2300, 900), (33, 128, 64, 9000, 40)])
def test_calls_repeat_bit_for_bit(t, B, page, D, prefix, own):
    """No result depends on when a copy lands or which CTA is first: the prefix kernel beside
    much and little memory traffic, one and two row tiles."""
    c = build_case([own - 7 * (i % 5) for i in range(B)], 1, None, 24, 12, D, page, HF, prefix)
    c["out_dt"] = HF
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, HF)
    first = None
    for _ in range(40):
        t.trit_attn_paged(job, err)
        torch.cuda.synchronize()
        first = (job.out.clone(), job.lse.clone()) if first is None else first
        assert torch.equal(first[0], job.out) and torch.equal(first[1], job.lse)
    assert int(err.item()) == 0 and bool(first[0].isfinite().all())
