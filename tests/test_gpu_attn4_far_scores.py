"""trit_attn_paged4 where scores are so large that 8 or 15 less of one (in powers of two) is no fp32 number.

All keys are alike, so that every score is the same fp32 number and every weight 1/n: out is the mean of the
values, to what test_gpu_attn4 derives for equal scores, (2 2^-11 + 2^-12) of the mean of
s c + |z| + 2^-16 (+ the output's rounding), and lse is score + ln n to 2^-20 of it (a
dozen roundings).  Lengths of several stages, one and many chunks."""
import math

import pytest

torch = pytest.importorskip("torch")

import prompt_ref as pr  # noqa: E402
import serving_ref as ref  # noqa: E402
from test_gpu_attn4 import BF, F32, HF, build_case, make_job, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,hq,hkv,dt", [(128, 8, 2, BF), (64, 16, 1, HF), (64, 3, 3, BF)])
def test_equal_far_scores(t, D, hq, hkv, dt, sign):  # noqa: F811
    lens, T = [1000, 130, 0, 5000], 2
    c = build_case(lens, T, None, hq, hkv, D, 16, dt)
    for b, n in enumerate(lens):
        pg, sl = ref.slots(c["table"][b], n, 16)
        k, s = (c["four"][i].permute(0, 2, 1, *range(3, c["four"][i].dim())) for i in (0, 2))
        k[pg, sl] = 0
        s[pg, sl] = torch.tensor([0.0, 1.0], dtype=torch.float16)
    c["q"] = torch.full_like(c["q"], 1024.0)         # q.k = 1024 D
    v = pr.values(c["four"][1], c["four"][3]).permute(0, 2, 1, 3)
    z = c["four"][3].double().permute(0, 2, 1, 3, 4)[..., 1].repeat_interleave(64, -1)
    # powers of two of the score about which 8, 15 or 16 less of it round, and far from there
    for e in (20.0, 23.9, 24.1, 26.7, 27.0000002, 27.0000005, 27.1, 27.3, 27.6, 27.9, 28.2, 29.3, 31.0, 60.0):
        scale = sign * 2.0 ** e * math.log(2.0) / (1024.0 * D)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = make_job(t, c, F32, scale)
        t.trit_attn_paged4(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        out, lse = job.out.double().cpu(), job.lse.double().cpu()
        exact = 1024.0 * D * float(torch.tensor(scale, dtype=torch.float32))
        for b, n in enumerate(lens):
            at = ref.slots(c["table"][b], n, 16)
            for i in range(T):
                see = n - T + i + 1
                if see <= 0:
                    assert not bool(out[b, i].any()) and bool((lse[b, i] == -math.inf).all())
                    continue
                vals, size = (x[at][:see].mean(0).repeat_interleave(hq // hkv, 0) for x in (v, (v - z).abs() + z.abs()))
                assert bool(((out[b, i] - vals).abs() <= (2.0 ** -10 + 2.0 ** -12) * size + 2.0 ** -16).all()), (e, b, i)
                assert bool(((lse[b, i] - exact - math.log(see)).abs() <= 2.0 ** -20 * abs(exact)).all()), (e, b, i)


def test_far_scores_that_grow(t):  # noqa: F811
    """Keys in rising steps across the same borders: only the greatest count."""
    n = 1600
    c = build_case([n], 1, None, 4, 1, 128, 16, HF, seed=2)
    pg, sl = ref.slots(c["table"][0], n, 16)
    k, s = (c["four"][i].permute(0, 2, 1, *range(3, c["four"][i].dim())) for i in (0, 2))
    k[pg, sl] = 0
    step = torch.arange(n) // 100
    s[pg, sl] = torch.stack((torch.zeros(n), 1.0 + step / 16), -1).half()[:, None, None]
    c["q"] = torch.full_like(c["q"], 1024.0)
    v = pr.values(c["four"][1], c["four"][3]).permute(0, 2, 1, 3)[pg, sl][-100:]
    z = c["four"][3].double().permute(0, 2, 1, 3, 4)[pg, sl][-100:, ..., 1].repeat_interleave(64, -1)
    v, size = v.mean(0), ((v - z).abs() + z.abs()).mean(0)
    for e in (22.5, 23.5, 26.6, 27.2, 27.9):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = make_job(t, c, F32, 2.0 ** e * math.log(2.0) / (1024.0 * 128))
        t.trit_attn_paged4(job, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert bool(((job.out[0, 0].double().cpu() - v).abs() <= (2.0 ** -10 + 2.0 ** -12) * size + 2.0 ** -16).all()), e
