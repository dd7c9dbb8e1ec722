"""trit_kv_append on the GPU against the formula in 64 bits, token by token.

Tolerance: the operator computes in fp32 and rounds once to the cache's type of
unit roundoff w (2^-8 bf16, 2^-11 fp16, subnormals of fp16 to 2^-25).  The
norm's sum of D squares carries at most (D + 6) 2^-24 relative error (half of
it through the root), a rotated column 3 roundings of each of its two
products; so |got - exact| <= w |exact| + (D + 12) 2^-24 (|a| + |b|) (1 + w) +
2^-25, |a| + |b| bounded by twice the vector's largest value."""
import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def t():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_plane_select_gb300 import build
    build.build()
    import bit_plane_select_gb300 as t
    torch.cuda.set_device(0)
    return t


def tables(top, rot):
    a = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return a.cos().float(), a.sin().float()


def run_case(t, lens, T, new, hq, hkv, D, rot, page, dt, src, norm, pairs, prefix=0, nhd=False, fused=False,
             seed=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages, pre, table = ref.make_batch(g, lens, T, page, prefix)
    shape = (pages, page, hkv, D) if nhd else (pages, hkv, page, D)
    kc, vc = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
    if nhd:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    width = (hq + 2 * hkv) * D
    qkv = (torch.randn((B * T, width), generator=g) * 3).to(src)
    cos, sin = tables(prefix + max(lens) + 1, rot) if rot else (None, None)
    gq, gk = (torch.rand(D, generator=g) + 0.5 for _ in range(2)) if norm else (None, None)
    eps = 1e-5

    def up(x):
        return None if x is None else x.cuda()
    dk = kc.cuda() if not nhd else kc.permute(0, 2, 1, 3).cuda().permute(0, 2, 1, 3)
    dv = vc.cuda() if not nhd else vc.permute(0, 2, 1, 3).cuda().permute(0, 2, 1, 3)
    parts = torch.split(qkv.cuda(), [hq * D, hkv * D, hkv * D], 1)
    if not fused:
        parts = [p.contiguous().view(B, T, -1, D) for p in parts]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dn = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    batch = t.KvBatch(table.cuda(), dl, T, new_lens=dn, prefix_table=up(pre), prefix_len=prefix)
    out = torch.full((B, T, hq, D), 7.0, dtype=dt, device="cuda")
    job = t.AppendJob(t.KvCache(dk, dv), batch, t.Rope(up(cos), up(sin), pairs, up(gq), up(gk), eps),
                      *parts, out)
    assert t.trit_kv_append(job, err) is out
    torch.cuda.synchronize()

    q, k, v = (p.view(B, T, -1, D).double() for p in torch.split(qkv, [hq * D, hkv * D, hkv * D], 1))
    wq = torch.zeros(B, T, hq, D, dtype=torch.float64)
    wk, wv = kc.double().clone(), vc.double().clone()
    for b in range(B):
        n = T if new is None else new[b]
        for i in range(n):
            own = lens[b] - n + i
            if own < 0:
                continue
            pg, sl = int(table[b, own // page]), own % page
            c, s = (cos[prefix + own].double(), sin[prefix + own].double()) if rot else (None, None)
            for h in range(hq):
                wq[b, i, h] = ref.rotate(ref.normed(q[b, i, h], gq, eps), c, s, rot, pairs)
            for h in range(hkv):
                wk[pg, h, sl] = ref.rotate(ref.normed(k[b, i, h], gk, eps), c, s, rot, pairs)
                wv[pg, h, sl] = v[b, i, h]
    w = UNIT[dt]
    for got, want in ((out.cpu(), wq), (dk.cpu(), wk), (dv.cpu(), wv)):
        big = 2 * want.abs().amax(-1, keepdim=True)
        tol = w * want.abs() + (D + 12) * 2.0 ** -24 * big * (1 + w) + 2.0 ** -25
        assert bool(((got.double() - want).abs() <= tol).all())
    return int(err.item()), out


BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # lens, T, new, hq, hkv, D, rot, page, cache, source, norm, pairs, prefix, nhd, fused
    ([1], 1, None, 20, 5, 128, 128, 64, BF, F32, False, False, 0, False, False),
    ([9, 1, 130], 1, None, 20, 5, 128, 128, 16, BF, F32, True, False, 77, False, True),
    ([7, 40, 16, 33], 5, [5, 0, 3, 1], 8, 2, 64, 64, 16, HF, F32, True, True, 0, True, False),
    ([7, 40, 16, 33], 5, [5, 0, 3, 1], 8, 2, 64, 48, 5, BF, BF, False, False, 1001, False, True),
    ([300], 300, None, 4, 4, 128, 72, 7, HF, HF, True, False, 0, False, False),
    ([12, 5], 3, None, 7, 7, 64, 24, 1, BF, F32, True, True, 3, True, True),
    ([12, 5], 3, None, 3, 1, 128, 0, 256, HF, F32, False, False, 0, False, False),
    ([65, 64], 2, [0, 0], 2, 1, 64, 64, 64, BF, F32, False, False, 0, False, False),
]


@pytest.mark.parametrize("case", CASES)
def test_append_matches_the_formula(t, case):
    err, _ = run_case(t, *case)
    assert err == 0


def test_padding_rows_are_zero(t):
    _, out = run_case(t, [7, 40], 4, [2, 0], 8, 2, 64, 64, 16, HF, F32, True, False)
    assert not bool(out[0, 2:].any()) and not bool(out[1].any())


def test_index_errors_are_flagged_and_nothing_is_written(t):
    """A new token before key 0, past the table, on a page outside the cache or at
    a position without a row in the tables: padding, and the flag."""
    g = torch.Generator().manual_seed(3)
    D, hkv, page, pages = 64, 2, 4, 6
    for lens, new, row, top in (([1], [3], [1, 2], 64), ([40], [1], [1, 2], 64), ([5], [1], [1, 6], 64),
                                ([5], [1], [1, -1], 64), ([8], [1], [1, 2], 7)):
        T = 3
        kc, vc = (torch.zeros(pages, hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
        cos, sin = (x.cuda() for x in tables(top, D))
        batch = t.KvBatch(torch.tensor([row], dtype=torch.int32, device="cuda"),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), T,
                          new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"))
        q, k, v = (torch.randn(1, T, h, D, generator=g).cuda() for h in (4, hkv, hkv))
        out = torch.ones(1, T, 4, D, dtype=BF, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        t.trit_kv_append(t.AppendJob(t.KvCache(kc, vc), batch, t.Rope(cos, sin), q, k, v, out), err)
        torch.cuda.synchronize()
        assert int(err.item()) == t.ERR_INDEX
        good = max(0, lens[0]) if new == [3] else 0      # [1] with 3 new tokens: the last one has a slot
        assert int((kc != 0).any(-1).any(1).sum()) == good
        assert int((out != 0).any(-1).any(-1).sum()) == good


def test_on_another_stream(t):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        err, _ = run_case(t, [9, 1, 130], 1, None, 20, 5, 128, 128, 16, BF, F32, True, False)
    assert err == 0
