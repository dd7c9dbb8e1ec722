"""Attention of prompts and behind a prefix where scores are so large that a step of fp32 there is many powers of two
of a weight: weights then stay within fp16's range, and equal scores have equal weights.

All keys are alike (or come in rising groups of which the last counts; behind a prefix the sequences' own are 0, of score
0, so that either kind counts alone): out is the mean of the values seen, to what
test_gpu_attn_prompt and test_gpu_attn_paged derive, (w + 2^-10 + 2^-12) of the mean of |v| (+ the output's
rounding + 2^-25; over 4 bits 2 2^-11 + 2^-12 of the mean of s c + |z|, + 2^-16), and lse is score + ln n to 2^-20 of it (a
dozen roundings)."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
import test_gpu_attn4 as four  # noqa: E402
import test_gpu_attn_paged as paged  # noqa: E402
import test_gpu_attn_prompt as prompt  # noqa: E402
from test_gpu_attn_paged import BF, F32, HF, UNIT, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu
# powers of two of the scores: about those where half a step passes what fp16 holds, and far from there
FAR = (20.0, 23.9, 24.1, 26.7, 27.0000002, 27.3, 27.9, 28.2, 28.7, 29.3, 30.6, 31.0, 33.3, 60.0)


def scale_of(e, D):
    """A scale that takes 1016 D to 2^e in powers of two, and the score that it gives."""
    scale = 2.0 ** e * math.log(2.0) / (1016.0 * D)
    return scale, 1016.0 * D * float(torch.tensor(scale, dtype=torch.float32))


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("nq,nk,hq,h,D,dt", [
    ([300], [300], 20, 5, 128, BF),              # a tile's blocks by turns
    ([300, 40], [700, 40], 8, 2, 64, HF),
    ([5], [400], 4, 4, 128, HF),
    ([1500, 700], [1500, 1100], 20, 5, 128, HF),  # a tile per CTA
    ([1500, 700], [1500, 1100], 20, 5, 64, BF),
])
def test_prompts(t, nq, nk, hq, h, D, dt, sign):  # noqa: F811
    c = prompt.build(nq, nk, hq, h, D, dt)
    first = [int(x) for x in c["ks"][:-1]]
    for a, n in zip(first, nk):
        c["k"][a:a + n] = 1.0
    c["q"] = torch.full_like(c["q"], sign * 1016.0)
    rising = dict(c, k=c["k"].clone())
    for a, n in zip(first, nk):
        group = torch.arange(n) // 100
        rising["k"][a:a + n] = (1.0 + sign * group / 64).to(dt)[:, None, None]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for e in FAR:
        scale, score = scale_of(e, D)
        for case in (c, rising):
            job = prompt.make(t, case, F32, scale)
            t.trit_attn_prompt(job, err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            for b, (n, m) in enumerate(zip(nq, nk)):
                rows = slice(int(c["qs"][b]), int(c["qs"][b]) + n)
                v = c["v"][first[b]:first[b] + m].double().repeat_interleave(hq // h, 1)
                see = torch.arange(n) + (m - n) + 1
                low = torch.zeros_like(see) if case is c else (see - 1) // 100 * 100
                if case is rising and e < 23:
                    continue
                sums = torch.cat((torch.zeros_like(v[:1]), v.cumsum(0)))
                sizes = torch.cat((torch.zeros_like(v[:1]), v.abs().cumsum(0)))
                count = (see - low).double()[:, None, None]
                want, mag = (sums[see] - sums[low]) / count, (sizes[see] - sizes[low]) / count
                out = job.out[rows].double().cpu()
                tol = (UNIT[dt] + 2.0 ** -10 + 2.0 ** -12) * mag + 2.0 ** -24 * want.abs() + 2.0 ** -25
                assert bool(((out - want).abs() <= tol).all()), (e, b, case is rising)
                if case is c:
                    lse = job.lse[rows].double().cpu()
                    assert bool(((lse - sign * score - count[:, 0].log()).abs() <= 2.0 ** -20 * score).all()), (e, b)


def check(c, job, v, size, w, floor, sign, score, e):
    out, lse = job.out.double().cpu(), job.lse.double().cpu()
    P, T = c["prefix"], c["T"]
    at = ref.slots(c["pre"], P, c["page"])
    for b, n in enumerate(c["lens"]):
        own = ref.slots(c["table"][b], n, c["page"])
        for i in range(T):
            see = max(0, n - T + i + 1)
            where, count, top = (at, P, score) if P and sign > 0 else (own, see, 0.0 if P else sign * score)
            if count == 0:
                continue
            want, mag = (x[where][:count].mean(0).repeat_interleave(c["hq"] // c["hkv"], 0) for x in (v, size))
            assert bool(((out[b, i] - want).abs() <= (w + 2.0 ** -10 + 2.0 ** -12) * mag + floor).all()), (e, b, i)
            assert bool(((lse[b, i] - top - math.log(count)).abs() <= 2.0 ** -20 * max(score, 1.0)).all()), (e, b, i)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("lens,T,hq,hkv,D,page,dt,prefix", [
    ([700, 33, 5000], 1, 20, 5, 128, 64, HF, 0),
    ([300, 9], 3, 8, 1, 64, 16, HF, 100),              # the prefix among the own keys
    ([70] * 30, 1, 8, 2, 128, 64, HF, 1000),           # on the tensor cores
    ([70] * 30, 1, 16, 2, 64, 16, BF, 1000),
])
def test_16_bit_cache(t, lens, T, hq, hkv, D, page, dt, prefix, sign):  # noqa: F811
    c = paged.build_case(lens, T, None, hq, hkv, D, page, dt, prefix)
    k = c["k"].permute(0, 2, 1, 3)
    for b, n in enumerate(lens):
        k[ref.slots(c["table"][b], n, page)] = 0.0 if prefix else 1.0
    k[ref.slots(c["pre"], prefix, page)] = 1.0
    c["q"] = torch.full_like(c["q"], 1016.0)
    v = c["v"].permute(0, 2, 1, 3).double()
    for e in FAR:
        scale, score = scale_of(e, D)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = paged.make_job(t, c, F32, scale=sign * scale)
        t.trit_attn_paged(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        check(c, job, v, v.abs(), UNIT[dt], 2.0 ** -25, sign, score, e)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_prefix_written_out_of_4_bits(t, sign):  # noqa: F811
    for lens, hq, hkv, D, prefix in (([70] * 60, 20, 5, 128, 3000), ([40] * 70, 16, 8, 64, 2500)):
        c = four.build_case(lens, 1, None, hq, hkv, D, 16, BF, prefix)
        where = [ref.slots(c["table"][b], n, 16) for b, n in enumerate(lens)] + [ref.slots(c["pre"], prefix, 16)]
        k, s = (c["four"][i].permute(0, 2, 1, *range(3, c["four"][i].dim())) for i in (0, 2))
        for at in where:
            k[at] = 0
            s[at] = torch.tensor([0.0, 1.0 if at is where[-1] else 0.0], dtype=torch.float16)
        c["q"] = torch.full_like(c["q"], 1016.0)
        v = pr.values(c["four"][1], c["four"][3]).permute(0, 2, 1, 3)
        z = c["four"][3].double().permute(0, 2, 1, 3, 4)[..., 1].repeat_interleave(64, -1)
        for e in FAR:
            scale, score = scale_of(e, D)
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            job = four.make_job(t, c, F32, sign * scale)
            t.trit_attn_paged4(job, err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            check(c, job, v, (v - z).abs() + z.abs(), 0.0, 2.0 ** -16, sign, score, e)
