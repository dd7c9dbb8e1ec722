"""One workspace under attention jobs of different sizes, in turn: zeroed once, and
every call leaves it ready for the next, whatever its batch, heads and prefix.  Each
call is checked against 64 bits with test_gpu_attn_paged's bound."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_attn_paged as base  # noqa: E402
from test_gpu_attn_paged import BF, HF, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu

JOBS = [
    # lens, T, new, hq, hkv, D, page, cache type, prefix, nhd
    ([1] * 256, 1, None, 4, 1, 64, 16, BF, 64, False),         # 257 sums of steps, prefix on the tensor cores
    ([3000], 1, None, 20, 5, 128, 64, BF, 0, False),           # one sequence over many CTAs
    ([900, 33, 700] * 11, 1, None, 8, 2, 64, 16, HF, 0, False),
    ([2, 30, 16, 1], 5, [2, 5, 0, 1], 6, 3, 64, 9, BF, 333, True),
    ([150, 131], 130, [130, 77], 8, 2, 64, 16, BF, 0, False),
    ([2000, 1], 1, None, 2, 1, 128, 16, HF, 0, False),
]


@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4, 5), (5, 4, 3, 2, 1, 0), (1, 5, 1, 2, 0, 2)])
def test_jobs_of_different_sizes_share_a_workspace(t, order):  # noqa: F811
    cases, jobs = {}, {}
    for i in set(order):
        lens, T, new, hq, hkv, D, page, dt, prefix, nhd = JOBS[i]
        c = base.build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=i)
        c["out_dt"] = dt
        cases[i], jobs[i] = c, base.make_job(t, c, dt)
    room = torch.zeros(max(j.workspace.numel() for j in jobs.values()), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    shared = {}
    for i, j in jobs.items():
        cache, batch, q, out, lse, _ = j._keep
        shared[i] = t.AttnJob(cache, batch, q, out, lse=lse, workspace=room)
    for i in order * 2:
        job = shared[i]
        job.out.fill_(7.0)
        job.lse.fill_(7.0)
        t.trit_attn_paged(job, err)
        torch.cuda.synchronize()
        base.check(cases[i], job.out, job.lse)
    assert int(err.item()) == 0
