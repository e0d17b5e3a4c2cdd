"""Limits of the paged cache's calls that the argument checks hold (CPU; the pointers are made up and no call here gets
past its checks)."""
import ctypes as C

import pytest

from tests.test_paged_host import A, INVALID, UNSUPPORTED, WORKSPACE, _cache, _desc, _seqs, ab  # noqa: F401


def _calls(ab, d, c, s, workspace):
    lib, view = ab._lib.load(), ab.attn_view_t(A, 0, 0, 0)  # (one row for all: sizes that no tensor of its own has)
    return [lib.paged_cache_write(C.byref(d), C.byref(c), C.byref(s), view, view, *workspace, None),
            lib.paged_cache_read(C.byref(d), C.byref(c), C.byref(s), view, view, *workspace, None),
            lib.sdpa_paged_fwd(C.byref(d), C.byref(c), C.byref(s), view, view, None, *workspace, None)]


@pytest.mark.parametrize("h,h_kv,rows", [(2, 2, 4), (8, 2, 8), (1, 1, 2), (40, 40, 80)])
@pytest.mark.parametrize("packed", [False, True])
def test_the_most_rows(ab, h, h_kv, rows, packed):  # noqa: F811
    """Rows (the new tokens times the larger of h and 2 h_kv) are counted in 32 bits, rounded up to blocks: the last ones
    that would leave that range are refused, those below come to the next check (of the workspace, left out here)."""
    for tokens, code in (((2 ** 31 - 1) // rows, UNSUPPORTED), ((2 ** 31 - 4096) // rows + 1, UNSUPPORTED),
                         ((2 ** 31 - 4096) // rows, WORKSPACE)):
        d = _desc(ab, b=1, h=h, h_kv=h_kv, s_q=1 if packed else tokens)
        s = _seqs(ab, **(dict(cu_new=A, tokens=tokens) if packed else {}))
        assert _calls(ab, d, _cache(ab), s, (None, 0)) == [code] * 3, tokens


NO_PLACES = [dict(scale_ss=0), dict(scale_sh=0), dict(scale_sp=0), dict(scale_sp=0, scale_ss=0, scale_sh=0), dict(ss=0), dict(sh=0),
             dict(sp=0)]


@pytest.mark.parametrize("kw", NO_PLACES, ids=str)
def test_a_write_needs_a_place_for_every_row_and_scale(ab, kw):  # noqa: F811
    """Strides of 0 (one scale for all rows, for one) are read through; a write would set one place from many rows at once."""
    c = _cache(ab, type=3, **kw)
    assert _calls(ab, _desc(ab), c, _seqs(ab), (None, 0)) == [INVALID, WORKSPACE, WORKSPACE]


def test_strides_along_what_there_is_one_of_may_be_anything(ab):  # noqa: F811
    one_page, one_head = dict(n_pages=1, sp=0, scale_sp=0), dict(sh=0, scale_sh=0)
    for c, d in ((_cache(ab, type=3, **one_page), _desc(ab)), (_cache(ab, type=3, **one_head), _desc(ab, h=1, h_kv=1)),
                 (_cache(ab, scale_ss=0, scale_sp=0, scale_sh=0), _desc(ab))):  # (a 16-bit cache has no scales)
        assert _calls(ab, d, c, _seqs(ab), (None, 0)) == [WORKSPACE] * 3
