"""Refusals of the position operators' calls: every check runs on the host before anything is launched, so
none of these needs a GPU.  The pointers are made up; no call here gets past its checks."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def ab():
    from attention_backward_02_gb300 import build
    build.build()
    import attention_backward_02_gb300 as ab
    ab._lib.load()
    return ab


OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5
A = 1 << 20  # an aligned address


def _qk(ab, **kw):
    base = dict(dtype=ab.ATTN_BF16, b=2, s=16, h=4, h_kv=2, d=128, rotary_dim=128, max_pos=64)
    base.update(kw)
    return ab.qk_norm_rope_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(h=0), OK), (dict(h_kv=0), OK), (dict(s=0), OK), (dict(rotary_dim=0, max_pos=0), OK),
    (dict(d=64, rotary_dim=16), OK), (dict(d=192, rotary_dim=176), OK),
    (dict(dtype=3), INVALID), (dict(b=0), INVALID), (dict(s=-1), INVALID), (dict(h=0, h_kv=0), INVALID),
    (dict(h=-1), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID), (dict(max_pos=0), INVALID),
    (dict(max_pos=1 << 31), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=1e-60), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(d=96, rotary_dim=0), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(b=1 << 20, s=1 << 12), UNSUPPORTED), (dict(b=1 << 40, s=1 << 40), UNSUPPORTED),
    (dict(b=1, s=1 << 28, h=32), UNSUPPORTED),
])
def test_qk_descriptor(ab, kw, code):
    f, b = C.c_size_t(), C.c_size_t()
    assert ab._lib.load().qk_norm_rope_workspace_size(C.byref(_qk(ab, **kw)), C.byref(f), C.byref(b)) == code
    if code == OK:
        assert f.value >= 4 and b.value > f.value


@pytest.mark.parametrize("field", ["interleaved", "weight_fp32"])
def test_qk_flags(ab, field):
    d = _qk(ab)
    setattr(d, field, 2)
    assert ab._lib.load().qk_norm_rope_workspace_size(C.byref(d), None, None) == INVALID


def _view(ab, ptr=A, sb=16 * 4 * 128, sh=128, ss=4 * 128):
    return ab.attn_view_t(ptr, sb, sh, ss)


def _fwd(ab, desc, ws=A, nbytes=1 << 30, **kw):
    a = dict(q=_view(ab), k=_view(ab), wq=A, wk=A, cos=A, sin=A, pos=A, yq=_view(ab), yk=_view(ab))
    a.update(kw)
    return ab._lib.load().qk_norm_rope_fwd(C.byref(desc), *a.values(), ws, nbytes, None)


def _bwd(ab, desc, ws=A, nbytes=1 << 30, **kw):
    v = _view(ab)
    a = dict(q=v, k=v, dyq=v, dyk=v, wq=A, wk=A, cos=A, sin=A, pos=A, dq=v, dk=v, dwq=A, dwk=A)
    a.update(kw)
    return ab._lib.load().qk_norm_rope_bwd(C.byref(desc), *a.values(), ws, nbytes, None)


def test_qk_calls(ab):
    d = _qk(ab)
    null, odd, stride = _view(ab, None), _view(ab, A + 8), _view(ab, ss=4 * 128 + 4)
    assert ab._lib.load().qk_norm_rope_fwd(None, *[_view(ab)] * 2, *[A] * 5, *[_view(ab)] * 2, A, 1 << 20, None) == NULLPTR
    for name in ("q", "k", "yq", "yk"):
        assert _fwd(ab, d, **{name: null}) == NULLPTR
        assert _fwd(ab, d, **{name: odd}) == ALIGN
        assert _fwd(ab, d, **{name: stride}) == ALIGN
    for name in ("q", "k", "dyq", "dyk", "dq", "dk"):
        assert _bwd(ab, d, **{name: null}) == NULLPTR
        assert _bwd(ab, d, **{name: odd}) == ALIGN
    for name in ("cos", "sin"):
        assert _fwd(ab, d, **{name: None}) == NULLPTR
        assert _fwd(ab, d, **{name: A + 4}) == ALIGN
    for name in ("wq", "wk"):
        assert _fwd(ab, d, **{name: A + 4}) == ALIGN
        assert _bwd(ab, d, **{name: A + 4}) == ALIGN
    for name in ("dwq", "dwk"):
        assert _bwd(ab, d, **{name: A + 2}) == ALIGN
    assert _fwd(ab, d, pos=A + 2) == ALIGN
    assert _fwd(ab, d, ws=None) == WORKSPACE and _fwd(ab, d, ws=A + 128) == WORKSPACE and _fwd(ab, d, nbytes=8) == WORKSPACE
    need = ab.qk_norm_rope_workspace_size(d)[1]
    assert _bwd(ab, d, nbytes=need - 1) == WORKSPACE
