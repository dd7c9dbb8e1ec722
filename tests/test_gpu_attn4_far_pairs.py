"""trit_attn_paged4 where the pairs (s, z) of V lie far apart.

What a row is off by follows its own keys.  A weight p (1 at the row's largest) of a term s c is off
by up to 2 2^-11 of itself or 2^-32, that of a term z by 2^-11 or 2^-40 (fp16's roundings, of numbers up to 2^15 and in units
of s within 2^8 of it; no s here is subnormal): with e and the sums' 2^-12 as test_gpu_attn4 derives them,
|out - exact| <= (2 2^-11 + 2 e + 2^-12) sum_j p_j (s c + |z|)_j + 2^-32 sum_j (s c + |z|)_j
(+ the output's rounding), however large another key's s is that carries no weight.  And what a
later token holds changes no bit of an earlier one's row."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
from test_gpu_attn4 import BF, F32, HF, UNIT, build_case, make_job, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def plain_keys(c, g, low):
    """Keys that are one number each, spread about 0, but for those in `low` ([sequence][index]), whose scores are 30
    below; queries of ones."""
    k, s = (c["four"][i].permute(0, 2, 1, *range(3, c["four"][i].dim())) for i in (0, 2))
    for b, n in enumerate(c["lens"]):
        pg, sl = ref.slots(c["table"][b], n, c["page"])
        z = 0.1 * torch.randn(n, generator=g)
        z[low[b]] = -30.0 / c["D"] ** 0.5
        k[pg, sl] = 0
        s[pg, sl] = torch.stack((torch.zeros(n), z), -1).half()[:, None, None]
    c["q"] = torch.ones_like(c["q"])


def set_values(c, b, s_of):
    """Values of sequence b: pairs (s, -7.5 s) with the given s [n] or [n, groups]."""
    n = c["lens"][b]
    pg, sl = ref.slots(c["table"][b], n, c["page"])
    s = s_of.half().float()
    if s.dim() == 1:
        s = s[:, None].expand(n, c["D"] // 64)
    c["four"][3].permute(0, 2, 1, 3, 4)[pg, sl] = torch.stack((s, -7.5 * s), -1).half()[:, None]


def check(c, out, out_dt):
    D, T = c["D"], c["T"]
    scale = D ** -0.5
    k, v = (pr.values(c["four"][i], c["four"][2 + i]).permute(0, 2, 1, 3) for i in (0, 1))
    z = c["four"][3].double().permute(0, 2, 1, 3, 4)[..., 1].repeat_interleave(64, -1)
    size = (v - z).abs() + z.abs()
    kz = c["four"][2].double()[..., 1].abs().nan_to_num(0).max()
    e = float(c["q"].double().abs().sum(-1).max() * kz) * scale * (D + 8) * 2.0 ** -24
    out = out.double().cpu()
    for b, n in enumerate(c["lens"]):
        at = ref.slots(c["table"][b], n, c["page"])
        new = T if c["new"] is None else c["new"][b]
        for i in range(new):
            see = n - new + i + 1
            if see <= 0:
                continue
            q = c["q"][b, i].double()
            want, _ = ref.attend(q, k[at][:see], v[at][:see], scale)
            mag, _ = ref.attend(q, k[at][:see], size[at][:see], scale)
            every = size[at][:see].sum(0).repeat_interleave(c["hq"] // c["hkv"], 0)
            tol = (2 * 2.0 ** -11 + 2 * e + 2.0 ** -12) * mag + 2.0 ** -32 * every + UNIT[out_dt] * want.abs()
            assert bool(((out[b, i] - want).abs() <= tol).all()), (b, i, float(((out[b, i] - want).abs() / tol).max()))


SHAPES = [
    # lens, T, new, Hq, heads, D, page, type
    ([700], 1, None, 4, 1, 128, 16, BF),
    ([700, 65, 3000], 1, None, 20, 5, 128, 64, HF),
    ([500, 33], 3, [3, 1], 8, 2, 64, 16, BF),
    ([300, 40], 6, [6, 5], 8, 2, 128, 16, HF),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("much", [100.0, 1000.0, 4000.0])
@pytest.mark.parametrize("little", [1e-3, 2e-4])
def test_weight_on_small_values_beside_a_large_one(t, shape, much, little):  # noqa: F811
    """A few keys of no weight have an s of 10^5 to 10^7 times the others'."""
    lens, T, new, hq, hkv, D, page, dt = shape
    c = build_case(lens, T, new, hq, hkv, D, page, dt, seed=int(much))
    g = torch.Generator().manual_seed(5)
    low = [torch.tensor(sorted({0, n // 3, n // 3 + 5, n - 17})) for n in lens]
    plain_keys(c, g, low)
    for b, n in enumerate(lens):
        s = little * (1 + 0.3 * torch.rand(n, D // 64, generator=g))
        s[low[b][:3]] = much
        s[low[b][3:], 0] = much / 10
        set_values(c, b, s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = make_job(t, c, F32)
    t.trit_attn_paged4(job, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(c, job.out, F32)


@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_all_through_a_stage(t, shape):  # noqa: F811
    """s from 10^-4 to 10^3 in scattered order, weights falling as s grows."""
    lens, T, new, hq, hkv, D, page, dt = shape
    c = build_case(lens, T, new, hq, hkv, D, page, dt, seed=7)
    g = torch.Generator().manual_seed(6)
    plain_keys(c, g, [torch.zeros(0, dtype=torch.long) for _ in lens])
    for b, n in enumerate(lens):
        s = 10.0 ** (-4 + 7 * torch.rand(n, generator=g) ** 3)
        pg, sl = ref.slots(c["table"][b], n, page)
        z = -torch.log(s) * 1.2 / D ** 0.5
        c["four"][2].permute(0, 2, 1, 3, 4)[pg, sl] = torch.stack((torch.zeros(n), z), -1).half()[:, None, None]
        set_values(c, b, s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out_dt in (F32, dt):
        job = make_job(t, c, out_dt)
        t.trit_attn_paged4(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        check(c, job.out, out_dt)


@pytest.mark.parametrize("lens,T,new,hq,hkv,D,page,dt", [
    ([200, 37, 6], 4, [4, 3, 4], 8, 2, 128, 16, BF),
    ([200, 37, 6], 4, [4, 3, 4], 8, 2, 64, 16, HF),
    ([150, 131], 100, [100, 70], 3, 3, 128, 64, HF),
    ([1000], 12, None, 20, 5, 128, 64, BF),
])
def test_a_later_token_changes_no_bit(t, lens, T, new, hq, hkv, D, page, dt):  # noqa: F811
    """The last token's key and value hold other numbers, of any size: the rows of the tokens before it are
    the same, bit by bit."""
    c = build_case(lens, T, new, hq, hkv, D, page, dt, seed=11)
    g = torch.Generator().manual_seed(8)
    for b, n in enumerate(lens):         # values of a few hundredths to some thousandths beside one another
        set_values(c, b, 10.0 ** (-3.5 + 2 * torch.rand(n, D // 64, generator=g)))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = make_job(t, c, F32)
    t.trit_attn_paged4(first, err)
    at = [ref.slots(c["table"][b], n, page) for b, n in enumerate(lens)]
    counts = [T if new is None else m for m in (new or [T] * len(lens))]
    for s, z in ((0.02, 1.0), (1.5, -9.0), (300.0, 0.0), (8000.0, -60000.0), (6e-8, 1e-7), (0.0, 5.0), (0.0, math.nan)):
        for (pg, sl), n in zip(at, lens):
            for i in (0, 1):
                c["four"][i].permute(0, 2, 1, 3)[pg[n - 1], sl[n - 1]] = torch.randint(256, (hkv, D // 2), generator=g, dtype=torch.uint8)
            c["four"][3].permute(0, 2, 1, 3, 4)[pg[n - 1], sl[n - 1]] = torch.tensor([s, z]).half()
        job = make_job(t, c, F32)
        t.trit_attn_paged4(job, err)
        torch.cuda.synchronize()
        for b, m in enumerate(counts):
            assert torch.equal(job.out[b, :m - 1], first.out[b, :m - 1]), (s, z, b)
            assert torch.equal(job.lse[b, :m - 1], first.lse[b, :m - 1]), (s, z, b)
    assert int(err.item()) == 0
