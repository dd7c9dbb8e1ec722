"""trit_draft_verify where no candidate is left, as its definition has it."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_draft_verify as verify  # noqa: E402
from test_gpu_draft_verify import t  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), -1.0])
def test_a_residual_whose_race_numbers_are_invalid_is_empty(t, bad):  # noqa: F811
    """The draw is over r where r is positive anywhere, even if no candidate is left: p does not
    step in."""
    for V in (203, 70000):
        p, q, draft, u, race = verify.inputs(4, 2, V, torch.float32, 11)
        u[:] = 0.999
        q[:2] = p[:2, :2]
        for b in range(2):                 # the residual is positive at one token, and its race number bad
            for k in range(2):
                x = int(draft[b, k])
                q[b, k, x] = 2 * p[b, k, x] + 1e-3      # not kept
                j = (x + 17) % V
                q[b, k, j] = 0.5 * p[b, k, j]
            race[b, (int(draft[b, 0]) + 17) % V] = bad
        assert verify.check(t, p, q, draft, u, race) == t.ERR_EMPTY
