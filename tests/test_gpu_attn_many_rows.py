"""trit_attn_paged at row counts whose products with D pass 31 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_attn_paged import BF, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_a_sequence_without_keys_is_zeroed_whole(t):  # noqa: F811
    """2^26 rows of D = 128 (2^31 vectors of four): every one 0, every lse -inf."""
    T, H, D = 1 << 16, 1 << 10, 128
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    k, v = (torch.zeros(2, H, 16, D, dtype=BF, device="cuda") for _ in range(2))
    q = torch.zeros(1, 1, H, D, dtype=BF, device="cuda").expand(1, T, H, D)
    out = torch.full((1, T, H, D), 7.0, dtype=BF, device="cuda")
    lse = torch.full((1, T, H), 7.0, device="cuda")
    batch = t.KvBatch(torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.zeros(1, dtype=torch.int32, device="cuda"), T)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.trit_attn_paged(t.AttnJob(t.KvCache(k, v), batch, q, out, lse=lse), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for part in out.view(64, -1):
        assert not bool(part.any())
    assert bool((lse == -math.inf).all())
    del out, lse
    torch.cuda.empty_cache()
