"""Packed rows of the paged cache's calls that belong to no sequence: whatever they hold, they are not written and change
nothing."""
import pytest

from tests.paged_problem import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("new", [(1, 2, 1), (40, 7, 90)])
def test_rows_of_no_sequence_change_nothing(cache, new):
    """Counts that begin behind the first rows and end before the last; those hold NaN, infinities or numbers."""
    import torch
    runs = []
    for other in (0.0, float("nan"), float("inf")):
        p = Problem("bfloat16", cache, [95, 60, 300], new, 8, 2, 128, extra_rows=21, seed=31)
        p.cu += 13
        rows = slice(13, 13 + sum(new))
        g = torch.Generator().manual_seed(32)
        def packed(heads):
            x = torch.full((p.rows, heads, 128), other, dtype=p.dt)
            x[rows] = torch.randn(sum(new), heads, 128, generator=g).to(p.dt)
            return x.cuda()
        k, v, q = packed(2), packed(2), packed(8)
        ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, k, v, cu_new=p.cu)
        assert p.ab.attn_query_status(ws) == 0
        back = [torch.full_like(k, 7) for _ in range(2)]
        p.ab.paged_cache_read(p.desc, p.cache, p.dtable, p.dlens, *back, cu_new=p.cu)
        o, lse = p.attend(q=q, o=torch.full_like(q, 7))
        for t in (*back, o):
            assert bool((t[:13] == 7).all()) and bool((t[13 + sum(new):] == 7).all()) and bool(t[rows].isfinite().all())
        assert bool(lse[:, :13].isnan().all()) and bool(lse[:, 13 + sum(new):].isnan().all())
        runs.append([t.view(torch.uint8) for t in (*p.cpool, *back, o[rows].contiguous(), lse[:, rows].contiguous())])
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], run))
