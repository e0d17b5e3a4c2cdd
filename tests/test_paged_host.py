"""The paged cache on the CPU: how the attention's work is shared out (a host program walks all shares of random
batches), the refusals of the calls (every check runs before anything is launched; the pointers are made up and no call
here gets past its checks), and the oracle's e4m3 numbers against torch's and closed forms."""
import ctypes as C
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

from oracle import paged as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5
A = 1 << 20  # an aligned address


def test_every_key_is_taken_once():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "paged_check")
        subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "attention_backward_02_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "paged_check.cu"), "-o", exe], check=True, capture_output=True, timeout=600)
        f = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout.split()
    got = dict(zip(f[::2], map(int, f[1::2])))
    assert got["batches"] > 10000 and got["pieces"] > 10 ** 6
    for k in ("holes", "twice", "empty", "slot", "chain", "heavy", "lanes"):
        assert got[k] == 0, got


# -------------------------------------------------------------------------------------------- oracle

def test_e4m3_numbers():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(P.E4M3)) and np.array_equal(want[~np.isnan(want)], P.E4M3[~np.isnan(want)])
    assert P.E4M3[0x7e] == 448 and P.E4M3[1] == 2.0 ** -9 and P.E4M3[8] == 2.0 ** -6
    # rounding: every number is its own code, ties go to the even code, beyond the largest stays there
    fine = [c for c in range(256) if c & 127 != 127]
    assert np.array_equal(P.to_code(P.E4M3[fine]), np.array(fine, np.uint8))
    for c in range(126):
        tie = (P.E4M3[c] + P.E4M3[c + 1]) / 2
        assert P.to_code(tie) == c + c % 2 and P.to_code(np.nextafter(tie, 0)) == c and P.to_code(np.nextafter(tie, 500)) == c + 1
    x = torch.randn(20000) * 100
    x = x[x.abs() < 448]
    assert np.array_equal(P.to_code(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert P.to_code(1e9) == 0x7e and P.to_code(-np.inf) == 0xfe and P.to_code(np.nan) & 127 == 127


def test_quantised_rows():
    code, sc = P.quantise(np.array([[0, 0, 0, 0], [448, -224, 1, 0], [np.inf, -2, 1, np.nan], [1e-38, 0, 0, 0]], np.float32))
    assert sc[0] == P.FLOOR / np.float32(448) and not code[0].any()
    assert sc[1] == 1 and np.array_equal(P.E4M3[code[1]], [448, -224, 1, 0])
    assert sc[2] == np.float32(2) / np.float32(448) and np.array_equal(P.E4M3[code[2]][:3], [448, -448, 224])
    assert code[2][3] & 127 == 127 and np.isfinite(sc).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    o, lse, p, *_ = P.attention(q * 0, k, v, 1.0, True)
    for i in range(3):  # equal scores: the mean of the first i + 3 values, log of their number
        assert np.allclose(o[i], v[:i + 3, 0].mean(0)) and np.allclose(lse[i], np.log(i + 3))
    o, lse, *_ = P.attention(q, k[:2], v[:2], 1.0, True)  # the first new token stands before the first key
    assert (o[0] == 0).all() and np.isinf(lse[0]).all() and np.allclose(o[1], v[0, 0])
    o, lse, *_ = P.attention(q, k, v, 0.5, False)
    s = np.einsum("mhd,nd->mhn", q, k[:, 0]) * 0.5
    w = np.exp(s) / np.exp(s).sum(-1, keepdims=True)
    assert np.allclose(o, w @ v[:, 0]) and np.allclose(lse, np.log(np.exp(s).sum(-1)))


# ------------------------------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def ab():
    from attention_backward_02_gb300 import build
    build.build()
    import attention_backward_02_gb300 as ab
    ab._lib.load()
    return ab


def _desc(ab, **kw):
    base = dict(dtype=ab.ATTN_BF16, b=2, h=8, h_kv=2, s_q=1, s_kv=1000, d=128, scale=0.1, mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    base.update(kw)
    return ab.sdpa_desc(**base)


def _cache(ab, **kw):
    base = dict(k=A, v=A, k_scale=A, v_scale=A, type=1, n_pages=50, page_size=64, sp=64 * 2 * 128, sh=128, ss=2 * 128,
                scale_sp=128, scale_sh=1, scale_ss=2)
    base.update(kw)
    return ab._lib.attn_paged_cache_t(*base.values())


def _seqs(ab, **kw):
    base = dict(page_table=A, table_stride=16, table_pages=16, lens=A, cu_new=None, tokens=0)
    base.update(kw)
    return ab._lib.attn_paged_seqs_t(*base.values())


SIZES = [
    (dict(), dict(), OK), (dict(dtype=0), dict(type=0), OK), (dict(dtype=0), dict(type=3), OK), (dict(mask=0), dict(), OK),
    (dict(s_kv=0), dict(n_pages=0), OK), (dict(s_q=0), dict(), OK), (dict(h=256), dict(), OK), (dict(d=64), dict(ss=128, sh=64), OK),
    (dict(dtype=3), dict(type=3), INVALID), (dict(dtype=0), dict(type=1), INVALID), (dict(), dict(type=2), INVALID),
    (dict(b=0), dict(), INVALID), (dict(h=9), dict(), INVALID), (dict(h_kv=0), dict(), INVALID), (dict(s_q=-1), dict(), INVALID),
    (dict(s_kv=-1), dict(), INVALID), (dict(scale=float("nan")), dict(), INVALID), (dict(mask=7), dict(), INVALID),
    (dict(), dict(n_pages=-1), INVALID), (dict(), dict(page_size=0), INVALID), (dict(), dict(ss=-256), INVALID),
    (dict(), dict(sp=-8), INVALID), (dict(), dict(type=3, scale_ss=-1), INVALID), (dict(), dict(type=3, scale_sh=1 << 31), UNSUPPORTED),
    (dict(mask=1), dict(), UNSUPPORTED), (dict(cu_seqlens_q=[1, 2], cu_seqlens_kv=[1, 2]), dict(), UNSUPPORTED),
    (dict(d=96), dict(), UNSUPPORTED), (dict(d=192), dict(), UNSUPPORTED), (dict(h=258, h_kv=2), dict(), UNSUPPORTED),
    (dict(b=65536), dict(), UNSUPPORTED), (dict(s_kv=(1 << 30) + 1), dict(), UNSUPPORTED), (dict(), dict(page_size=8), UNSUPPORTED),
    (dict(), dict(page_size=48), UNSUPPORTED), (dict(), dict(page_size=512), UNSUPPORTED), (dict(), dict(n_pages=1 << 31), UNSUPPORTED),
    (dict(), dict(ss=1 << 26), UNSUPPORTED), (dict(), dict(sh=1 << 31), UNSUPPORTED), (dict(), dict(sp=1 << 38), UNSUPPORTED),
    (dict(), dict(ss=260), ALIGN), (dict(), dict(sh=132), ALIGN), (dict(), dict(sp=12), ALIGN), (dict(), dict(type=3, sh=136), ALIGN),
]


@pytest.mark.parametrize("dk,ck,code", SIZES, ids=lambda x: str(x).replace(" ", "")[:40])
def test_sizes(ab, dk, ck, code):
    lib, n = ab._lib.load(), C.c_size_t()
    d, c = _desc(ab, **dk), _cache(ab, **ck)
    for fn in (lib.paged_cache_workspace_size, lib.sdpa_paged_workspace_size):
        assert fn(C.byref(d), C.byref(c), C.byref(n)) == code
        if code == OK:
            assert n.value >= 256 and n.value % 256 == 0
            assert fn(C.byref(d), C.byref(c), None) == NULLPTR
    assert lib.sdpa_paged_workspace_size(None, C.byref(c), C.byref(n)) == NULLPTR
    assert lib.paged_cache_workspace_size(C.byref(d), None, C.byref(n)) == NULLPTR


CALLS = [
    (dict(), dict(k=None), dict(), NULLPTR), (dict(), dict(v=None), dict(), NULLPTR), (dict(), dict(type=3, k_scale=None), dict(), NULLPTR),
    (dict(), dict(type=3, v_scale=None), dict(), NULLPTR), (dict(), dict(), dict(page_table=None), NULLPTR),
    (dict(), dict(), dict(lens=None), NULLPTR), (dict(), dict(k=A + 8), dict(), ALIGN), (dict(), dict(v=A + 2), dict(), ALIGN),
    (dict(), dict(type=3, v_scale=A + 2), dict(), ALIGN), (dict(), dict(), dict(lens=A + 1), ALIGN),
    (dict(), dict(), dict(page_table=A + 2), ALIGN), (dict(), dict(), dict(cu_new=A + 2), ALIGN),
    (dict(), dict(), dict(table_pages=15), INVALID), (dict(), dict(), dict(table_stride=-1), INVALID),
    (dict(), dict(), dict(cu_new=A, tokens=-1), INVALID), (dict(), dict(), dict(cu_new=A, tokens=1 << 28), UNSUPPORTED),
    (dict(s_q=1 << 30), dict(), dict(), UNSUPPORTED), (dict(d=96), dict(), dict(), UNSUPPORTED),
]


@pytest.mark.parametrize("dk,ck,sk,code", CALLS, ids=lambda x: str(x).replace(" ", "")[:40])
def test_calls_refuse(ab, dk, ck, sk, code):
    lib, view = ab._lib.load(), ab.attn_view_t(A, 8 * 128, 128, 8 * 128)
    d, c, s = _desc(ab, **dk), _cache(ab, **ck), _seqs(ab, **sk)
    for fn in (lib.paged_cache_write, lib.paged_cache_read):
        assert fn(C.byref(d), C.byref(c), C.byref(s), view, view, A, 1 << 40, None) == code
    assert lib.sdpa_paged_fwd(C.byref(d), C.byref(c), C.byref(s), view, view, A, A, 1 << 40, None) == code


def test_views_and_workspaces(ab):
    lib, view = ab._lib.load(), ab.attn_view_t(A, 8 * 128, 128, 8 * 128)
    d, c, s = _desc(ab), _cache(ab), _seqs(ab)
    null, odd, stride = (ab.attn_view_t(*x) for x in ((None, 1024, 128, 1024), (A + 8, 1024, 128, 1024), (A, 1024, 132, 1024)))
    for bad, code in ((null, NULLPTR), (odd, ALIGN), (stride, ALIGN)):
        for pair in ((bad, view), (view, bad)):
            for fn in (lib.paged_cache_write, lib.paged_cache_read):
                assert fn(C.byref(d), C.byref(c), C.byref(s), *pair, A, 1 << 40, None) == code
            assert lib.sdpa_paged_fwd(C.byref(d), C.byref(c), C.byref(s), *pair, None, A, 1 << 40, None) == code
    for fn in (lib.paged_cache_write, lib.paged_cache_read):
        assert fn(C.byref(d), C.byref(c), None, view, view, A, 1 << 40, None) == NULLPTR
        for ws, n in ((None, 1 << 40), (A + 128, 1 << 40), (A, 255)):
            assert fn(C.byref(d), C.byref(c), C.byref(s), view, view, ws, n, None) == WORKSPACE
    need = C.c_size_t()
    lib.sdpa_paged_workspace_size(C.byref(d), C.byref(c), C.byref(need))
    for ws, n in ((None, 1 << 40), (A + 128, 1 << 40), (A, need.value - 1)):
        assert lib.sdpa_paged_fwd(C.byref(d), C.byref(c), C.byref(s), view, view, None, ws, n, None) == WORKSPACE
    assert lib.sdpa_paged_fwd(C.byref(d), C.byref(c), C.byref(s), view, view, A + 2, A, 1 << 40, None) == ALIGN


def test_the_binding_refuses(ab):
    torch = pytest.importorskip("torch")
    kv = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(v=kv.half()), dict(v=kv[:3]), dict(v=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16).transpose(1, 2)),
                dict(k=kv.float(), v=kv.float()), dict(k=kv[..., ::2], v=kv[..., ::2])):
        with pytest.raises(ValueError):
            ab.paged_cache(**dict(dict(k=kv, v=kv), **bad))
    eight = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.zeros(4, 16, 2)
    for bad in (dict(), dict(k_scale=sc), dict(k_scale=sc.double(), v_scale=sc), dict(k_scale=sc[:, :8], v_scale=sc[:, :8])):
        with pytest.raises(ValueError):
            ab.paged_cache(eight, eight, **bad)
    cache, d = ab.paged_cache(kv, kv), _desc(ab, d=64, s_kv=64)
    with pytest.raises(ValueError):  # not CUDA tensors
        ab.paged_cache_write(d, cache, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), kv, kv)


class _Memory:
    """A CUDA tensor as the argument checks see it."""

    def __init__(self, ptr, dtype, shape, stride=None, device=0):
        self.ptr, self.dtype, self.shape, self.index = ptr, dtype, tuple(shape), device
        self.strides, self.device = stride, f"cuda:{device}"

    def data_ptr(self):
        return self.ptr

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        if self.strides is None:
            s, n = [], 1
            for x in reversed(self.shape):
                s.insert(0, n)
                n *= x
            self.strides = tuple(s)
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def numel(self):
        return 1 << 40


def _fakes(torch, **kw):
    """(a descriptor's cache, and the arguments of a call) of made-up CUDA tensors."""
    m = lambda dt, *shape, ptr=A: _Memory(ptr, dt, shape, device=kw.get("device", 0))
    bf, i32, e4 = torch.bfloat16, torch.int32, torch.float8_e4m3fn
    pool = [m(e4, 50, 64, 2, 128, ptr=A * (i + 1)) for i in range(2)]
    size = [m(torch.float32, 50, 64, 2, ptr=A * (i + 3)) for i in range(2)]
    return pool, size, dict(table=m(i32, 2, 16), lens=m(i32, 2), q=m(bf, 2, 8, 1, 128), kv=m(bf, 2, 2, 1, 128))


def test_a_cache_whose_memory_was_replaced(ab):
    """tensor.data = ... gives pages other memory, strides and type: a call reads what the tensors are then, and refuses
    what no longer fits together."""
    import types
    torch = pytest.importorskip("torch")
    pool, size, t = _fakes(torch)
    cache = ab.paged_cache(*pool, k_scale=size[0], v_scale=size[1])
    stream = types.SimpleNamespace(cuda_stream=0, device=types.SimpleNamespace(index=0))
    call = lambda: ab._paged_call("call", _desc(ab), cache, t["table"], t["lens"], None, 0, stream)
    call()
    assert (cache.k, cache.v, cache.k_scale, cache.type, cache.n_pages, cache.ss, cache.scale_ss) == (A, 2 * A, 3 * A, 3, 50, 256, 2)
    pool[0].ptr, size[1].ptr = 7 * A, 9 * A
    call()
    assert (cache.k, cache.v_scale) == (7 * A, 9 * A)
    for x in pool:
        x.dtype, x.shape, x.strides = torch.bfloat16, (60, 64, 2, 128), (1 << 20, 512, 128, 1)
    call()
    assert (cache.type, cache.n_pages, cache.sp, cache.ss, cache.sh) == (1, 60, 1 << 20, 512, 128)
    for name, value in (("dtype", torch.float16), ("shape", (60, 64, 2, 64)), ("strides", (1 << 20, 256, 128, 1)), ("index", 1)):
        old = getattr(pool[1], name)
        setattr(pool[1], name, value)
        with pytest.raises(ValueError):
            call()
        setattr(pool[1], name, old)
    call()


@pytest.mark.parametrize("name,kw", [
    ("table", dict(index=1)), ("lens", dict(index=1)), ("table", dict(shape=(3, 16))), ("lens", dict(shape=(3,))),
    ("table", dict(strides=(32, 2))), ("q", dict(index=1)), ("q", dict(shape=(2, 4, 1, 128))), ("kv", dict(index=1)),
    ("kv", dict(shape=(2, 2, 2, 128)))])
def test_tensors_of_another_device_or_shape_are_refused(ab, name, kw):
    torch = pytest.importorskip("torch")
    import types
    pool, size, t = _fakes(torch)
    cache = ab.paged_cache(*pool, k_scale=size[0], v_scale=size[1])
    for k, v in kw.items():
        setattr(t[name], k, v)
    stream = types.SimpleNamespace(cuda_stream=0, device=types.SimpleNamespace(index=0))
    with pytest.raises(ValueError):
        if name == "kv":
            ab.paged_cache_write(_desc(ab), cache, t["table"], t["lens"], t["kv"], t["kv"], workspace=_Memory(A, torch.uint8, (1,)),
                                 stream=stream)
        else:
            ab.sdpa_paged_fwd(_desc(ab), cache, t["table"], t["lens"], t["q"], t["q"], workspace=_Memory(A, torch.uint8, (1,)),
                              stream=stream)


def test_calls_run_on_the_pages_device_and_their_workspace_on_the_stream(ab, monkeypatch):
    """With the tensors on device 1 and device 0 current: the device is made current for the call, the stream is that of
    device 1, and a workspace that the call makes is memory of the stream it is given.  torch and the launches are stood in for."""
    import contextlib
    import types
    torch = pytest.importorskip("torch")
    current, made, seen, at = [0], [], [], [None]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    @contextlib.contextmanager
    def use(stream):
        before, at[0] = at[0], stream
        yield
        at[0] = before

    def empty(n, dtype, device):
        made.append(at[0])
        return _Memory(A, dtype, (n,), device=1)

    names = ("float16", "bfloat16", "float32", "int32", "uint8", "float8_e4m3fn", "device")
    raw = types.SimpleNamespace(_cuda_getDevice=lambda: current[0], _cuda_getCurrentRawStream=lambda d: 100 + d)
    fake = types.SimpleNamespace(empty=empty, _C=raw, **{n: getattr(torch, n) for n in names},
                                 cuda=types.SimpleNamespace(stream=use, device=device))
    real = ab._lib.load()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real, name)
            return lambda *a: seen.append((name, current[0], a[-1])) or 0

    pool, size, t = _fakes(torch, device=1)
    cache = ab.paged_cache(*pool, k_scale=size[0], v_scale=size[1])
    monkeypatch.setattr(ab, "_torch_module", fake)
    monkeypatch.setattr(ab._lib, "load", Lib)
    stream = types.SimpleNamespace(cuda_stream=5, device=types.SimpleNamespace(index=1))
    args = (_desc(ab), cache, t["table"], t["lens"])
    for i, (fn, x) in enumerate(((ab.paged_cache_write, t["kv"]), (ab.paged_cache_read, t["kv"]), (ab.sdpa_paged_fwd, t["q"]))):
        fn(*args, x, x)
        fn(*args, x, x, stream=stream)
        assert made[-2] is None and made[-1] is stream and seen[-2:] == [(fn.__name__, 1, 101), (fn.__name__, 1, 5)], i
        with pytest.raises(ValueError):  # a stream of another device
            fn(*args, x, x, stream=types.SimpleNamespace(cuda_stream=5, device=types.SimpleNamespace(index=0)))
    assert current == [0]
