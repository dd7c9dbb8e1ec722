"""trit_attn_prompt where sequences have more queries than keys: the rows that see no key are 0, and -inf
in lse, whatever was there (outputs start as 7; tolerances as test_gpu_attn_prompt derives them).

The search for a tile by length counts a sequence's units with at least so many key blocks; the deficits lie on both
sides of 127 + a unit (128 tokens over the query heads of a key head), past which the first units have
fewer than no blocks by that count."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_attn_prompt import BF, F32, HF, build, check, make, run, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu

CASES = [
    # queries, keys, Hq, heads, D, type
    ([300, 40], [10, 40], 20, 5, 128, BF),
    ([5, 400], [5, 100], 8, 2, 128, HF),
    ([700, 5], [0, 5], 8, 2, 64, BF),
    ([159, 3], [1, 3], 4, 1, 128, BF),
    ([160, 3], [0, 3], 4, 1, 128, BF),
    ([161, 3], [1, 3], 4, 1, 64, HF),
    ([192, 3], [0, 3], 4, 1, 128, HF),
    ([255, 90], [0, 3], 3, 3, 64, BF),
    ([400, 290], [17, 1], 3, 3, 128, BF),
    ([1500, 700, 1], [200, 1300, 0], 24, 8, 64, BF),              # tiles by length, a few an SM
    ([90, 41, 0, 0, 500], [0, 0, 0, 7, 200], 21, 3, 64, HF),
    ([300, 2], [20, 0], 130, 1, 64, BF),
    ([(i * 53) % 260 for i in range(32)], [(i * 97) % 130 for i in range(32)], 4, 2, 128, HF),
    # found in their order: one sequence, many, and many tiles
    ([600], [10], 20, 5, 128, BF),
    ([(i * 53) % 260 for i in range(33)], [(i * 97) % 130 for i in range(33)], 4, 2, 64, BF),
    ([1900, 1400], [800, 100], 24, 8, 64, HF),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_rows_without_keys_are_zero(t, case, wide):  # noqa: F811
    nq, nk, hq, h, D, dt = case
    err, _ = run(t, build(nq, nk, hq, h, D, dt, seed=D + len(nq)), F32 if wide else dt)
    assert err == 0


@pytest.mark.parametrize("many", [False, True])
def test_starts_that_fall(t, many):  # noqa: F811
    """The sequences before the fall are whole, the ones behind it that have rows of theirs are left out (`many`:
    found in their order)."""
    c = build([20, 480], [20, 480], 8, 2, 64, BF)
    at = torch.tensor([2, 22, 502, 102, 482] + [482] * (30 if many else 0))
    job = make(t, dict(c, qs=at, ks=at), BF)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        t.trit_attn_prompt(job, err)
    torch.cuda.synchronize()
    assert int(err.item()) == t.ERR_INDEX
    check(c, job)
