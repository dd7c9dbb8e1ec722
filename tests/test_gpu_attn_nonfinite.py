"""Infinities and NaN in K and V of keys that a row must not see.

Token t of a sequence sees own keys 0..i; a later token's K or V of inf or NaN (an
overflow of the 16-bit cache, say) changes nothing of it, and rows that see no key
give 0 and -inf whatever the cache holds.  Rows that do see such a V have the
definition's non-finite value in its columns and test_gpu_attn_paged's bound in the
others."""
import math

import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
import test_gpu_attn_paged as base  # noqa: E402
from test_gpu_attn_paged import BF, F32, HF, UNIT, t  # noqa: E402,F401

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan

CASES = [
    # lens, T, new, hq, hkv, D, page, cache type, prefix, nhd
    ([9, 40, 8], 4, [4, 2, 3], 8, 2, 64, 16, HF, 0, False),            # an item in one CTA; padding rows
    ([9, 40, 8], 4, [4, 2, 0], 20, 5, 128, 16, BF, 0, False),
    ([20, 64], 2, None, 2, 2, 128, 7, BF, 0, True),                    # 8 rows, pages that end inside a tile
    ([3000, 5], 8, [8, 3], 20, 5, 128, 16, BF, 0, False),              # an item over many CTAs
    ([2500, 700], 3, [3, 2], 8, 2, 64, 32, HF, 0, False),
    ([150, 131], 130, [130, 77], 8, 2, 64, 16, BF, 0, False),          # many row tiles
    ([2, 30, 16, 6], 5, [2, 5, 0, 1], 20, 5, 128, 16, BF, 1005, False),   # a prefix on the tensor cores
    ([2, 30, 16, 6], 5, [2, 5, 0, 1], 6, 3, 64, 9, BF, 333, True),     # and on the other path
    ([700 + i for i in range(34)], 3, [1 + i % 3 for i in range(34)], 8, 1, 128, 128, HF, 1111, False),
]


def plant(c, what):
    """Bad values at the own keys of new tokens: {(sequence, own key): column of V or -1 for K}."""
    at = {}
    k, v = (x.permute(0, 2, 1, 3) for x in (c["k"], c["v"]))
    for b, n in enumerate(c["lens"]):
        new = c["T"] if c["new"] is None else c["new"][b]
        for i in {1, new - 1}:
            if not 1 <= i < new or n - new + i < 0:
                continue
            own = n - new + i
            pg, sl = (int(x[own]) for x in ref.slots(c["table"][b], n, c["page"]))
            if what == "k":
                k[pg, sl, :, 3] = NAN if i == 1 else INF
            else:
                v[pg, sl, :, (5 + 7 * i) % c["D"]] = {"inf": INF, "-inf": -INF, "nan": NAN}[what]
            at[b, own] = i
        if what != "k" and new < c["T"] and n > new + 2:      # an old key, beside padding rows
            pg, sl = (int(x[1]) for x in ref.slots(c["table"][b], n, c["page"]))
            v[pg, sl, :, 2] = INF
    return at


@pytest.mark.parametrize("what", ["inf", "-inf", "nan", "k"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_only_the_rows_that_see_a_bad_key_change(t, case, wide, what):  # noqa: F811
    lens, T, new, hq, hkv, D, page, dt, prefix, nhd = case
    c = base.build_case(lens, T, new, hq, hkv, D, page, dt, prefix, nhd, seed=7 + prefix)
    at = plant(c, what)
    assert at
    out_dt = F32 if wide else dt
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    job = base.make_job(t, c, out_dt)
    t.trit_attn_paged(job, err)
    t.trit_attn_paged(job, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    out, lse = job.out.double().cpu(), job.lse.double().cpu()
    k, v = (x.permute(0, 2, 1, 3).double() for x in (c["k"], c["v"]))
    slots = ref.slots(c["pre"], prefix, page)
    pk, pv = k[slots], v[slots]
    w, wo = UNIT[dt], UNIT[out_dt]
    for b, n in enumerate(lens):
        slots = ref.slots(c["table"][b], n, page)
        keys, vals = torch.cat((pk, k[slots])), torch.cat((pv, v[slots]))
        m = T if new is None else new[b]
        for i in range(T):
            if i >= m:
                assert not bool(out[b, i].any()) and bool((lse[b, i] == -INF).all()), (b, i)
                continue
            own = max(0, n - m + i + 1)
            if what == "k" and any((b, j) in at for j in range(own)):
                assert bool(out[b, i].isnan().all())      # a NaN or infinite score among those seen
                continue
            see = prefix + own
            q = c["q"][b, i].double()
            want, wl = ref.attend(q, keys[:see], vals[:see], D ** -0.5)
            good = want.isfinite()
            assert bool(torch.equal(want.isnan(), out[b, i].isnan())), (b, i)
            assert bool((want[want.isinf()] == out[b, i][want.isinf()]).all()), (b, i)
            mag, _ = ref.attend(q, keys[:see], vals[:see].abs().nan_to_num(0, 0, 0), D ** -0.5)
            tol = (w + 2.0 ** -10 + 2.0 ** -12) * mag + wo * want.abs() + 2.0 ** -25
            assert bool(((out[b, i] - want).abs()[good] <= tol[good]).all()), (b, i)
            assert bool(((lse[b, i] - wl).abs() <= 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -22 * wl.abs()).all()), (b, i)
