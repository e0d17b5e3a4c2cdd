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


def _bias(ab, **kw):
    base = dict(table=A, table_type=2, num_buckets=32, max_distance=128, bidirectional=1)
    base.update(kw)
    return ab.attn_relbias_t(*base.values())


def _sdpa(ab, **kw):
    base = dict(dtype=ab.ATTN_F16, b=2, h=4, h_kv=2, s_q=64, s_kv=96, d=64, scale=0.125)
    base.update(kw)
    return ab.sdpa_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(num_buckets=2, max_distance=2, bidirectional=0), OK), (dict(num_buckets=128), OK),
    (dict(num_buckets=4, max_distance=2), OK), (dict(max_distance=65536), OK), (dict(table_type=0), OK),
    (dict(num_buckets=1, bidirectional=0), INVALID), (dict(num_buckets=2), INVALID), (dict(num_buckets=7), INVALID),
    (dict(num_buckets=0), INVALID), (dict(num_buckets=-4), INVALID), (dict(max_distance=8), INVALID),
    (dict(max_distance=16, bidirectional=0), INVALID), (dict(max_distance=-1), INVALID), (dict(table_type=3), INVALID),
    (dict(table_type=-1), INVALID), (dict(bidirectional=2), INVALID), (dict(num_buckets=130), UNSUPPORTED),
    (dict(max_distance=65537), UNSUPPORTED),
])
def test_relbias_descriptor(ab, kw, code):
    f, b, n = C.c_size_t(), C.c_size_t(), C.c_int64()
    lib, bias, desc = ab._lib.load(), _bias(ab, **kw), _sdpa(ab)
    assert lib.sdpa_relbias_workspace_size(C.byref(desc), C.byref(bias), C.byref(f), C.byref(b)) == code
    assert lib.attn_relbias_bucket(C.byref(bias), -5, C.byref(n)) == code
    if code == OK:
        plain = ab.sdpa_workspace_size(desc)
        assert f.value > plain[0] and b.value > plain[1]


def test_relbias_buckets(ab):
    """Against the integer definition, over every border."""
    from oracle import position as P
    for nb, far, both in [(32, 128, 1), (32, 128, 0), (64, 1024, 0), (128, 1000, 1), (16, 100, 1), (2, 2, 0), (4, 9, 1),
                          (3, 5, 0), (5, 77, 0), (128, 2000, 0)]:
        bias = _bias(ab, num_buckets=nb, max_distance=far, bidirectional=both)
        for delta in range(-far - 5, far + 6):
            assert ab.relbias_bucket(bias, delta) == P.bucket(delta, nb, far, bool(both)), (nb, far, both, delta)
        for delta in (-2 ** 63, 2 ** 63 - 1):
            assert ab.relbias_bucket(bias, delta) == P.bucket(delta, nb, far, bool(both))
    assert ab._lib.load().attn_relbias_bucket(None, 0, C.byref(C.c_int64())) == NULLPTR
    assert ab._lib.load().attn_relbias_bucket(C.byref(_bias(ab)), 0, None) == NULLPTR


def test_relbias_calls(ab):
    lib, desc = ab._lib.load(), _sdpa(ab)
    v = ab.attn_view_t(A, 4 * 96 * 64, 64, 256)
    fwd = lambda b=None, d=desc, views=(v,) * 4, lse=A, ws=A, n=1 << 30: lib.sdpa_relbias_fwd_stats(
        C.byref(d), None if b == 0 else C.byref(b or _bias(ab)), *views, lse, ws, n, None)
    bwd = lambda b=None, d=desc, views=(v,) * 8, lse=A, dt=A, ws=A, n=1 << 30: lib.sdpa_relbias_bwd(
        C.byref(d), None if b == 0 else C.byref(b or _bias(ab)), *views[:5], lse, *views[5:], dt, ws, n, None)
    assert lib.sdpa_relbias_workspace_size(None, C.byref(_bias(ab)), None, None) == NULLPTR
    assert lib.sdpa_relbias_workspace_size(C.byref(desc), None, None, None) == NULLPTR
    for call, views in ((fwd, 4), (bwd, 8)):
        assert call(0) == NULLPTR and call(_bias(ab, table=None)) == NULLPTR and call(lse=None) == NULLPTR
        assert call(_bias(ab, table=A + 2)) == ALIGN and call(_bias(ab, table=A + 1, table_type=0)) == ALIGN
        assert call(_bias(ab, num_buckets=7)) == INVALID
        assert call(d=_sdpa(ab, d=96)) == UNSUPPORTED and call(d=_sdpa(ab, b=1, h=65536, h_kv=1)) == UNSUPPORTED
        for i in range(views):
            bad = [v] * views
            bad[i] = ab.attn_view_t(None, 4 * 96 * 64, 64, 256)
            assert call(views=bad) == NULLPTR
            bad[i] = ab.attn_view_t(A + 8, 4 * 96 * 64, 64, 256)
            assert call(views=bad) == ALIGN
        need = ab.sdpa_relbias_workspace_size(desc, _bias(ab))[call is bwd]
        assert call(ws=None) == WORKSPACE and call(ws=A + 16) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert bwd(dt=None) == NULLPTR and bwd(dt=A + 2) == ALIGN


def test_decode_refusals(ab):
    lib = ab._lib.load()
    size = lambda d, b=None: lib.sdpa_relbias_decode_workspace_size(C.byref(d), C.byref(b or _bias(ab)), C.byref(C.c_size_t()))
    base = dict(s_q=1, s_kv=4096, mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    ok = _sdpa(ab, **base)
    assert size(ok) == OK and size(_sdpa(ab, **{**base, "s_kv": 0})) == OK
    assert size(_sdpa(ab, **{**base, "s_q": 2})) == INVALID and size(_sdpa(ab, **{**base, "mask": 0})) == INVALID
    assert size(_sdpa(ab, **{**base, "mask": 1})) == INVALID and size(ok, _bias(ab, num_buckets=3)) == INVALID
    assert size(_sdpa(ab, **{**base, "d": 192})) == UNSUPPORTED
    assert size(_sdpa(ab, **{**base, "s_kv": 1 << 31, "b": 1, "h_kv": 1})) == UNSUPPORTED
    packed = _sdpa(ab, **base, cu_seqlens_q=[1, 2], cu_seqlens_kv=[10, 30])
    assert size(packed) == UNSUPPORTED
    assert lib.sdpa_relbias_decode_workspace_size(C.byref(ok), C.byref(_bias(ab)), None) == NULLPTR
    v = ab.attn_view_t(A, 4096 * 128, 64, 128)
    call = lambda i=None, x=None, lens=A, b=None, ws=A, n=1 << 30: lib.sdpa_relbias_decode(
        C.byref(ok), C.byref(b or _bias(ab)), *[x if j == i else v for j in range(3)], lens, x if i == 3 else v, ws, n, None)
    for i in range(4):
        assert call(i, ab.attn_view_t(None, 0, 64, 128)) == NULLPTR
        assert call(i, ab.attn_view_t(A + 8, 0, 64, 128)) == ALIGN and call(i, ab.attn_view_t(A, 4, 64, 128)) == ALIGN
    assert call(lens=A + 2) == ALIGN and call(b=_bias(ab, table=None)) == NULLPTR
    assert call(ws=None) == WORKSPACE and call(ws=A + 8) == WORKSPACE and call(n=300) == WORKSPACE


def test_relbias_buckets_next_to_a_border(ab):
    """Distances that come within 1e-9 of a border (as the logarithms count) without reaching it, and their
    neighbours; and borders that are whole numbers."""
    from oracle import position as P
    near = [(32, 43921, 16325), (64, 23785, 10409), (32, 61179, 36534), (64, 16463, 13545), (73, 905, 347),
            (99, 5217, 1067), (126, 58181, 42031), (127, 32736, 22146), (128, 65536, 65535)]
    for nb, far, x in near:
        for both in ([0, 1] if 2 * nb <= 128 else [0]):
            n = 2 * nb if both else nb
            bias = _bias(ab, num_buckets=n, max_distance=far, bidirectional=both)
            for delta in (-x - 1, -x, 1 - x, x - 1, x, x + 1):
                assert ab.relbias_bucket(bias, delta) == P.bucket(delta, n, far, bool(both)), (n, far, both, delta)
    for nb, far, whole in [(128, 65536, 2048), (64, 65536, 1 << 12), (8, 65536, 1 << 9)]:
        e = nb // 2
        bias = _bias(ab, num_buckets=nb, max_distance=far, bidirectional=0)
        for delta in (-whole, 1 - whole, -e, -far, 1 - far):
            assert ab.relbias_bucket(bias, delta) == P.bucket(delta, nb, far, False), (nb, far, delta)


def test_relbias_buckets_at_drawn_borders(ab):
    """Every border of drawn layouts up to the largest: the last distance below it and the first at it, found by
    bisection of the integer definition."""
    import random
    from oracle import position as P
    rng = random.Random(17)
    for _ in range(60):
        nb = rng.randint(2, 128)
        far = rng.randint(nb // 2 + 1, 65536)
        bias = _bias(ab, num_buckets=nb, max_distance=far, bidirectional=0)
        for n in range(nb // 2 + 1, nb):
            lo, hi = nb // 2, far  # bucket(lo) < n or lo is the border; bucket(hi) >= n
            while lo < hi:
                mid = (lo + hi) // 2
                if P.bucket(-mid, nb, far, False) >= n:
                    hi = mid
                else:
                    lo = mid + 1
            for x in (lo - 1, lo):
                assert ab.relbias_bucket(bias, -x) == P.bucket(-x, nb, far, False), (nb, far, x)


def test_lse_shape(ab):
    """lse is taken in the documented order of its elements alone: [B, h, S_q] (packed: [h, T_q]), its neighbouring
    dimensions merged or not, and refused where another order has the same number of elements."""
    import types
    import torch
    call = types.SimpleNamespace(where="call", device=-1, refuse=ab._Call.refuse.__get__(
        types.SimpleNamespace(where="call", device=-1)))
    take = lambda d, shape, t: ab._lse_ptr(call, d, t, shape)
    fixed, want = _sdpa(ab), (2, 4, 64)
    for shape in [(2, 4, 64), (2, 4, 64, 1), (512,), (8, 64), (2, 256), (1, 2, 4, 64)]:
        t = torch.zeros(shape)
        assert take(fixed, want, t) == t.data_ptr()
    for shape in [(2, 64, 4), (4, 2, 64), (64, 8), (2, 64, 4, 1), (2, 4, 32), (2, 4, 65), (511,), (2, 4, 8, 8)]:
        with pytest.raises(ValueError, match="lse"):
            take(fixed, want, torch.zeros(shape))
    for t in (torch.zeros(2, 64, 4).permute(0, 2, 1), torch.zeros(2, 4, 64, dtype=torch.float64)):
        with pytest.raises(ValueError, match="lse"):
            take(fixed, want, t)
    packed = _sdpa(ab, cu_seqlens_q=[30, 50], cu_seqlens_kv=[30, 50])
    for shape in [(4, 50), (200,), (4, 50, 1)]:
        t = torch.zeros(shape)
        assert take(packed, None, t) == t.data_ptr()
    for shape in [(50, 4), (2, 4, 25), (4, 51)]:
        with pytest.raises(ValueError, match="lse"):
            take(packed, None, torch.zeros(shape))
    empty = _sdpa(ab, s_q=0)
    for shape in [(2, 4, 0), (0,)]:
        take(empty, (2, 4, 0), torch.zeros(shape))


class _Memory:
    """A CUDA tensor as the argument checks see it."""

    def __init__(self, ptr, dtype, shape, contiguous=True, device=0):
        self.ptr, self.dtype, self.shape, self.contiguous, self.index = ptr, dtype, shape, contiguous, device
        self.device = f"cuda:{device}"

    def data_ptr(self):
        return self.ptr

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index


def test_a_table_whose_memory_was_replaced(ab):
    """tensor.data = ... gives a table other memory and another type: a call reads what the tensor is then."""
    import types
    import torch
    stream = types.SimpleNamespace(cuda_stream=0, device=types.SimpleNamespace(index=0))
    table = _Memory(A, torch.float32, (32, 4))
    bias = ab.relbias(table)
    assert (bias.table, bias.table_type, bias.num_buckets) == (A, 2, 32)
    table.ptr, table.dtype, table.shape = 3 * A, torch.bfloat16, (16, 4)
    ab._relbias_call("call", _sdpa(ab), bias, table, stream)
    assert (bias.table, bias.table_type, bias.num_buckets) == (3 * A, 1, 16)
    for bad in (dict(dtype=torch.float64), dict(shape=(16, 5)), dict(shape=(64,)), dict(contiguous=False)):
        table = _Memory(A, torch.float32, (32, 4))
        bias = ab.relbias(table)
        for k, v in bad.items():
            setattr(table, k, v)
        with pytest.raises(ValueError, match="table"):
            ab._relbias_call("call", _sdpa(ab), bias, _Memory(A, torch.float32, (2, 4, 64)), stream)
    with pytest.raises(ValueError, match="table"):
        ab._relbias_call("call", _sdpa(ab), ab.relbias(_Memory(A, torch.float32, (32, 4), device=1)),
                         _Memory(A, torch.float32, (2, 4, 64)), stream)


def test_a_workspace_made_by_a_call_is_memory_of_its_stream(ab, monkeypatch):
    """Every call that makes its own workspace takes it from the stream it is given: the current stream's free
    memory may still be in use by work queued there.  torch and the library's launches are stood in for."""
    import contextlib
    import types
    import torch
    made, at = [], [None]

    @contextlib.contextmanager
    def use(stream):
        before, at[0] = at[0], stream
        yield
        at[0] = before

    def empty(n, dtype, device):
        made.append(at[0])
        return types.SimpleNamespace(data_ptr=lambda: A, numel=lambda: n, record_stream=lambda s: None)

    raw = types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda d: 0)
    names = ("float16", "bfloat16", "float32", "int32", "uint8", "device")
    now = types.SimpleNamespace(cuda_stream=0)
    fake = types.SimpleNamespace(empty=empty, _C=raw, **{n: getattr(torch, n) for n in names}, cuda=types.SimpleNamespace(
        stream=use, current_stream=lambda *a: now, current_device=lambda: 0))
    real = ab._lib.load()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name) if name.endswith("_size") else lambda *a: 0

    d, bias = _sdpa(ab), ab.relbias(_Memory(A, torch.float32, (32, 4)))
    one = _sdpa(ab, s_q=1, s_kv=4096, mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    n = ab.nsa_desc(dtype=ab.ATTN_BF16, cu_seqlens_q=[64], cu_seqlens_kv=[128], n1=4, n2=1, d=128, scale=0.1,
                    block_size=64, block_count=2, sparse_mode=0)
    v, x, lse = ab.attn_view_t(A, 4 * 96 * 64, 64, 256), _Memory(A, torch.float32, (8,)), _Memory(A, torch.float32, (2, 4, 64))
    dt = _Memory(A, torch.float32, (32, 4))
    calls = [lambda **k: ab.sdpa_fwd_stats(d, v, v, v, v, lse, **k),
             lambda **k: ab.sdpa_bwd(d, v, v, v, v, v, lse, v, v, v, **k),
             lambda **k: ab.nsa_selected_attn_fwd(n, *[x] * 7, **k),
             lambda **k: ab.nsa_selected_attn_bwd(n, *[x] * 11, **k),
             lambda **k: ab.nsa_block_lists(n, x, x, x, **k),
             lambda **k: ab.sdpa_relbias_fwd_stats(d, bias, v, v, v, v, lse, **k),
             lambda **k: ab.sdpa_relbias_bwd(d, bias, v, v, v, v, v, lse, v, v, v, dt, **k),
             lambda **k: ab.sdpa_relbias_decode(one, bias, v, v, v, None, v, **k),
             lambda **k: ab.qk_norm_rope_fwd(_qk(ab, rotary_dim=0), v, v, None, None, None, None, v, v, **k),
             lambda **k: ab.qk_norm_rope_bwd(_qk(ab, rotary_dim=0), v, v, v, v, None, None, None, None, v, v, **k)]
    monkeypatch.setattr(ab, "_torch_module", fake)
    monkeypatch.setattr(ab._lib, "load", Lib)
    stream = types.SimpleNamespace(cuda_stream=5, device=types.SimpleNamespace(index=0))
    for i, call in enumerate(calls):
        call()
        call(stream=stream)
        assert len(made) == 2 * i + 2 and made[-2] is None and made[-1] is stream, i


def test_status_of_a_workspace_on_another_device(ab, monkeypatch):
    """The status is read behind the current stream of the workspace's device, with that device current.  torch and the
    library are stood in for."""
    import contextlib
    import types
    import torch
    current, seen = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    fake = types.SimpleNamespace(cuda=types.SimpleNamespace(
        device=device, current_stream=lambda d=None: types.SimpleNamespace(cuda_stream=100 + (current[0] if d is None else d))))

    def query(ws, stream, flags):
        seen.append((current[0], ws.value, stream.value))
        flags._obj.value = 2
        return 7

    monkeypatch.setattr(ab, "_torch_module", fake)
    monkeypatch.setattr(ab._lib, "load", lambda: types.SimpleNamespace(attn_query_status=query))
    for index in (0, 1):
        assert ab.attn_query_status(_Memory(A, torch.uint8, (256,), device=index)) == 2
        assert ab.attn_query_status(_Memory(A, torch.uint8, (256,), device=index), types.SimpleNamespace(cuda_stream=7)) == 2
    assert seen == [(0, A, 100), (0, A, 7), (1, A, 101), (1, A, 7)] and current == [0]
