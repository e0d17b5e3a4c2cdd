"""sdpa_relbias_bwd where every CTA has several work units, so that what one leaves behind (bucket sums, the running
sum of one bucket, ring and barrier phases, zeroed rows of a packed tile, fp32 shares of dK and dV) meets the next.
Against the fp64 definition within the bounds of the biased backward's tests, and bit for bit between runs."""
import numpy as np
import pytest

from tests.test_gpu_relbias import Problem

pytestmark = pytest.mark.gpu

SMS = 152


def _shares(p):
    """Units that share the query heads of a (key tile, kv head): by the size of their sums in the workspace, which the
    ordered mode does not have."""
    size = lambda mode: p.ab.sdpa_relbias_workspace_size(_desc(p, mode), p.bias)[1]
    one = 2 * p.tk * p.hk * p.d * 4
    return max(1, round((size(0) - size(2)) / one))


def _desc(p, mode):
    d = type(p.desc).from_buffer_copy(p.desc)
    d.deterministic = mode
    return d


CASES = [
    # dtype, lens, h, hk, d, mask, shares, kw
    ("float16", [(500, 500)], 40, 40, 64, 0, 1, dict(b=2)),
    ("bfloat16", [(500, 470)], 40, 40, 128, 2, 1, dict(b=2, layout="bhsd")),
    ("float16", [(300, 300), (129, 200), (0, 70), (511, 400), (64, 64), (257, 513)], 30, 30, 64, 2, 1, {}),
    ("bfloat16", [(190, 260), (333, 333), (70, 1), (130, 390), (1, 129)], 36, 36, 128, 0, 1, {}),
    ("float16", [(130, 900)], 64, 8, 64, 1, 4, {}),
    ("bfloat16", [(260, 130)], 64, 8, 64, 2, 4, dict(b=4)),
    ("bfloat16", [(400, 520), (130, 260), (0, 40), (333, 700)], 32, 4, 128, 2, 4, {}),
]


@pytest.mark.parametrize("dtype,lens,h,hk,d,mask,shares,kw", CASES)
def test_several_units_a_cta(dtype, lens, h, hk, d, mask, shares, kw):
    p = Problem(dtype, lens, h, hk, d, mask, 32, 128, True, seed=d + h + mask, **kw)
    got = _shares(p)
    assert got == shares
    assert sum((n + 127) // 128 for _, n in p.lens) * hk * got > 1.5 * SMS
    o, lse = p.inputs_bwd()
    first = p.bwd(o, lse)
    p.check_bwd(first, o, lse)
    again = p.bwd(o, lse)
    for i in (1, 2, 3):  # (dQ: atomic adds)
        np.testing.assert_array_equal(first[i], again[i])


@pytest.mark.parametrize("dtype,lens,h,d,mask,mode,splits,kw", [
    ("float16", [(640, 640)], 40, 64, 2, 1, 2, dict(b=2)),          # units of two and three key tiles, two a CTA
    ("bfloat16", [(300, 700), (513, 257)], 36, 128, 0, 1, 2, {}),
    ("float16", [(500, 500)], 40, 64, 0, 2, 0, dict(b=2)),
    ("bfloat16", [(300, 300), (129, 200), (0, 70), (511, 400)], 36, 128, 2, 2, 0, {}),
])
def test_several_units_a_cta_in_the_reproducible_modes(dtype, lens, h, d, mask, mode, splits, kw):
    p = Problem(dtype, lens, h, h, d, mask, 32, 128, False, seed=d + h + mode, mode=mode, **kw)
    p.desc.dq_splits = splits
    o, lse = p.inputs_bwd()
    first = p.bwd(o, lse)
    p.check_bwd(first, o, lse)
    for a, b in zip(first, p.bwd(o, lse)):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("dtype,lens,h,hk,d,mask,kw", [
    ("float16", [(1 + 7 * n % 40, 1 + 11 * n % 37) for n in range(256)], 18, 18, 64, 2, {}),  # the most packed sequences
    ("bfloat16", [(33, 20)], 18, 18, 128, 0, dict(b=256)),
])
def test_more_units_than_the_host_plans(dtype, lens, h, hk, d, mask, kw):
    """More units than a plan holds: they are taken in turn.  Forward and backward, the forward's units past its estimate's
    reach too."""
    import torch
    p = Problem(dtype, lens, h, hk, d, mask, 32, 128, True, seed=d, **kw)
    assert sum((n + 127) // 128 for _, n in p.lens) * hk > 4096
    o, lse = p.fwd()
    ot, lt = torch.from_numpy(o).to(p.dt), lse.astype(np.float32)
    first, again = p.bwd(ot, lt), p.bwd(ot, lt)
    for i in (1, 2, 3):
        np.testing.assert_array_equal(first[i], again[i])
    pick = [0, h - 1]  # the definition takes a few of the heads
    few = Problem(dtype, lens, 2, 2, d, mask, 32, 128, True, **kw)
    few.q, few.k, few.v, few.do = (t[:, pick] for t in (p.q, p.k, p.v, p.do))
    few.table = p.table[:, pick].contiguous()
    few.check_fwd(o[:, pick], lse[:, pick])
    few.check_bwd([x[:, pick] for x in first], ot[:, pick], lt[:, pick])
