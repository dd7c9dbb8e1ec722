"""trit_draft_verify on the GPU against a plain implementation, sequence by
sequence: whole numbers, equal (the definition names its fp32 roundings: one
product, one difference, one quotient)."""
import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_plane_select_gb300 import build
    build.build()
    import bit_plane_select_gb300 as t
    torch.cuda.set_device(0)
    return t


def inputs(B, T, V, dtype, seed, alpha=0.7, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.softmax(sharp * torch.randn(B, T + 1, V, generator=g), -1)
    r = torch.softmax(sharp * torch.randn(B, T, V, generator=g), -1)
    q = (alpha * p[:, :T] + (1 - alpha) * r).to(dtype)
    p = p.to(dtype)
    draft = torch.multinomial(q.float().reshape(B * T, V), 1, generator=g).reshape(B, T).to(torch.int32)
    u = torch.rand(B, T, generator=g)
    race = torch.empty(B, V).exponential_(generator=g)
    return p, q, draft, u, race


def check(t, p, q, draft, u, race, n=None, pad=0, twice=True):
    B, T, V = q.shape

    def strided(x):
        if not pad:
            return x.cuda()
        room = torch.full(x.shape[:-1] + (V + pad,), float("nan"), dtype=x.dtype, device="cuda")
        room[..., :V] = x.cuda()
        return room[..., :V]
    tokens = torch.full((B, T + 1), 99, dtype=torch.int32, device="cuda")
    accepted = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nd = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    job = t.VerifyJob(strided(p), strided(q), draft.cuda(), u.cuda(), strided(race), tokens, accepted, n_draft=nd)
    for _ in range(2 if twice else 1):
        t.trit_draft_verify(job, err)
    torch.cuda.synchronize()
    for b in range(B):
        nb = T if n is None else min(max(n[b], 0), T)
        want, k = ref.verify(p[b], q[b], draft[b], u[b], race[b], nb)
        assert tokens[b].tolist() == want and int(accepted[b]) == k, b
    return int(err.item())


@pytest.mark.parametrize("B,T,V,dtype,pad", [
    (1, 1, 1, torch.float32, 0), (3, 2, 2, torch.float32, 1), (5, 4, 37, torch.float32, 0),
    (1, 4, 32000, torch.float32, 0), (7, 3, 50257, torch.float32, 0), (4, 8, 4096, torch.bfloat16, 8),
    (9, 33, 130, torch.float16, 0), (2, 70, 999, torch.float32, 3), (300, 1, 65, torch.bfloat16, 0),
    (2, 3, 70000, torch.float32, 0), (25, 2, 65541, torch.float16, 3), (30, 1, 66000, torch.bfloat16, 0)])
def test_matches_the_plain_form(t, B, T, V, dtype, pad):
    for seed, alpha in ((1, 0.5), (2, 0.97)):
        x = inputs(B, T, V, dtype, seed, alpha)
        assert check(t, *x, pad=pad) == 0
        n = [(3 * b + seed) % (T + 1) for b in range(B)]
        assert check(t, *x, n=n, pad=pad) == 0


def test_the_edges(t):
    """u = 0; equal distributions (the residual is empty: p decides); zero
    probabilities; ties; zero, infinite and NaN race numbers and probabilities."""
    p, q, draft, u, race = inputs(8, 3, 203, torch.float32, 5)
    u[0] = 0.0                                              # all kept
    q[1] = p[1, :3]
    u[1] = 0.9999999                                        # may be lost by rounding: p then decides
    p[2, 0, draft[2, 0].long()] = 0.0                       # a token the target never takes
    p[3] = 0.0
    p[3, :, 7] = 1.0                                        # one candidate
    q[4, 0] = 0.0                                           # the draft gives its own token no weight
    race[5, 10:20] = 0.0                                    # infinite quotients: the lowest wins
    race[6, :100] = float("inf")
    race[6, 150] = float("nan")
    p[7, :, 11] = float("nan")
    q[7, :, 12] = float("nan")
    assert check(t, p, q, draft, u, race) == 0
    race[:] = 1.0
    p[:, :, 50:60] = p[:, :, 50:51].clone()                 # equal quotients
    q[:, :, 50:60] = q[:, :, 50:51].clone()
    assert check(t, p, q, draft, u, race) == 0
    p[:] = float("nan")
    assert check(t, p, q, draft, u, race) == t.ERR_EMPTY


def test_bad_indexes_are_flagged(t):
    p, q, draft, u, race = inputs(3, 4, 77, torch.float32, 6)
    draft[0, 1] = 77
    draft[1, 0] = -5
    assert check(t, p, q, draft, u * 0, race) == t.ERR_INDEX
    p, q, draft, u, race = inputs(3, 4, 77, torch.float32, 7)
    assert check(t, p, q, draft, u, race, n=[9, -1, 2]) == t.ERR_INDEX


def test_small_probabilities(t):
    """Subnormal quotients and products keep their order."""
    p, q, draft, u, race = inputs(4, 2, 4099, torch.float32, 8)
    p *= 1e-38
    q *= 1e-38
    assert check(t, p, q, draft, u, race) == 0
    race *= 1e-30
    assert check(t, p, q, draft, u, race) == 0
