"""Attention of prompts where scores are so large that a step of fp32 there is many powers of two
of a weight: weights then stay within fp16's range, and equal scores have equal weights.

All keys are alike (or come in rising groups of which the last counts): out is the mean of the values seen, to what
test_gpu_attn_prompt derives, (w + 2^-10 + 2^-12) of the mean of |v| (+ the output's rounding + 2^-25), and lse is score +
ln n to 2^-20 of it (a dozen roundings)."""
import math

import pytest

torch = pytest.importorskip("torch")

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
