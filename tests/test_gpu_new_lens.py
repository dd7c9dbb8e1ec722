"""New lengths outside their range, given to the serving operators that read them."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_attn_paged as attn  # noqa: E402
from test_gpu_attn_paged import BF, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 40, 700])
def test_new_lens_outside_their_range_are_flagged(t, prefix):  # noqa: F811
    """Clamped to [0, T], and the flag, by both operators that read them."""
    for lens in ([30, 40], [30, 40] * 9):
        c = attn.build_case(lens, 4, [9, -2] * (len(lens) // 2), 8, 2, 64, 16, BF, prefix)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        job = attn.make_job(t, c, BF)
        t.trit_attn_paged(job, err)
        torch.cuda.synchronize()
        c["out_dt"], c["new"] = BF, [4, 0] * (len(lens) // 2)
        attn.check(c, job.out, job.lse)
        assert int(err.item()) == t.ERR_INDEX


def test_append_flags_new_lens_outside_their_range(t):  # noqa: F811
    D, T = 64, 3
    for n, good in ((7, T), (-1, 0)):
        kc, vc = (torch.zeros(4, 2, 16, D, dtype=BF, device="cuda") for _ in range(2))
        batch = t.KvBatch(torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"),
                          torch.tensor([20], dtype=torch.int32, device="cuda"), T,
                          new_lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        q, k, v = (torch.randn(1, T, h, D, device="cuda") for h in (4, 2, 2))
        out = torch.ones(1, T, 4, D, dtype=BF, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        t.trit_kv_append(t.AppendJob(t.KvCache(kc, vc), batch, t.Rope(), q, k, v, out), err)
        torch.cuda.synchronize()
        assert int(err.item()) == t.ERR_INDEX
        assert int((kc != 0).any(-1).any(1).sum()) == good and int((out != 0).any(-1).any(-1).sum()) == good
