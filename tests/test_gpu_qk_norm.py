"""GPU parity of qk_norm_rope_fwd / _bwd with the fp64 definition, through the C ABI.

Bounds.  u = 2^-24 (fp32 half step), h = eps(type) / 2 (output half step).  Forward: the mean square sums at
most 24 terms in a lane and three shuffles, all positive, so its relative error is below 30 u and r's below
16 u; x r w adds 2 u, the turn (one product, one fused product) 2 u of |a| + |b|, cos and sin being inputs:
    |err| <= h |y| + 32 u (|a| + |b|) + tiny,
where tiny is half the type's smallest subnormal.  Backward: xh and dz carry 18 u and 2 u, g one more, the mean
of g xh at most 30 u of the mean of |g xh|, and the last two operations 2 u:
    |err| <= h |dx| + 64 u r (|g| + |xh| mean|g xh|) + tiny,   |g| from |dz| <= |dy_a| + |dy_b|.
Weight gradient: a sum of n = tokens x heads products, each within 24 u, in any order within n u:
    |err| <= (n + 64) u sum|dz xh|."""
import numpy as np
import pytest

from oracle import position as P
from tests import harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


def _name(dt):
    return str(dt).split(".")[-1]


class Problem:
    """Inputs on the GPU, and fp64 copies, of one call.  layout: 'bshd', 'bhsd' or 'pad' (token-major with
    eight spare elements behind every head and a spare head behind every token)."""

    def __init__(self, dtype, b, s, h, hk, d, rot, interleaved=False, weights="16", positions="random",
                 layout="bshd", seed=0, max_pos=97, size=1.0):
        import torch
        import attention_backward_02_gb300 as ab
        self.ab, self.torch = ab, torch
        self.dt = torch.float16 if dtype == "float16" else torch.bfloat16
        self.b, self.s, self.h, self.hk, self.d, self.rot, self.inter = b, s, h, hk, d, rot, interleaved
        self.eps, self.max_pos, self.layout = 1e-5, max_pos, layout
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *sh: torch.randn(*sh, generator=g)
        self.x = [self.place((rnd(b, s, n, d) * size).to(self.dt)) for n in (h, hk)]
        self.dy = [self.place(rnd(b, s, n, d).to(self.dt)) for n in (h, hk)]
        wt = {"16": self.dt, "32": torch.float32, "none": None}[weights]
        self.w = [None if wt is None else (1 + 0.3 * rnd(d)).to(wt).cuda() for _ in range(2)]
        self.cos = self.sin = self.pos = None
        if rot:
            ang = rnd(max_pos, rot // 2) * 3
            self.cos, self.sin = ang.cos().cuda(), ang.sin().cuda()
            if positions == "random":
                self.pos = torch.randint(0, max_pos, (b, s), generator=g, dtype=torch.int32).cuda()
        self.desc = ab.qk_norm_rope_desc(dtype=ab.ATTN_F16 if dtype == "float16" else ab.ATTN_BF16, b=b, s=s, h=h,
                                         h_kv=hk, d=d, rotary_dim=rot, interleaved=interleaved, eps=self.eps,
                                         weight_fp32=weights == "32", max_pos=max_pos if rot else 0)

    def place(self, t):
        """t [b, s, n, d] as a [b, n, s, d] CUDA tensor in this problem's layout."""
        b, s, n, d = t.shape
        if self.layout == "bhsd":
            return t.cuda().permute(0, 2, 1, 3).contiguous()
        if self.layout == "pad":
            buf = self.torch.full((b, s, n + 1, d + 8), 7.0, dtype=t.dtype, device="cuda")
            buf[:, :, :n, :d] = t.cuda()
            return buf[:, :, :n, :d].permute(0, 2, 1, 3)
        return t.cuda().permute(0, 2, 1, 3)

    def new(self, k):
        return self.place(self.torch.full((self.b, self.s, (self.h, self.hk)[k], self.d), float("nan"), dtype=self.dt))

    def f64(self, t):
        return t.permute(0, 2, 1, 3).double().cpu().numpy()

    def angles(self):
        if not self.rot:
            return None, None
        if self.pos is None:
            rows = np.broadcast_to(np.arange(self.s), (self.b, self.s))
        else:
            rows = self.pos.cpu().numpy()
        return self.cos.double().cpu().numpy()[rows], self.sin.double().cpu().numpy()[rows]

    def weight(self, k):
        return np.ones(self.d) if self.w[k] is None else self.w[k].double().cpu().numpy()

    def fwd(self, out=None, **kw):
        out = out or [self.new(0), self.new(1)]
        ws = self.ab.qk_norm_rope_fwd(self.desc, *self.x, *self.w, self.cos, self.sin, *out, positions=self.pos, **kw)
        return out, ws

    def bwd(self, out=None, dw=None, **kw):
        out = out or [self.new(0), self.new(1)]
        dw = dw or [self.torch.full((self.d,), float("nan"), device="cuda") for _ in range(2)]
        ws = self.ab.qk_norm_rope_bwd(self.desc, *self.x, *self.dy, *self.w, self.cos, self.sin, *out, *dw,
                                      positions=self.pos, **kw)
        return out, dw, ws

    def check_fwd(self, out):
        cos, sin = self.angles()
        for k in range(2):
            x, w = self.f64(self.x[k]), self.weight(k)
            if x.size == 0:
                continue
            ref = P.norm_rope(x, w, self.eps, cos, sin, self.rot, self.inter)
            z = np.abs(P.norm_rope(x, w, self.eps, None, None, 0, False))
            mag = z + self.partner(z)
            n = _name(self.dt)
            err = np.abs(self.f64(out[k]) - ref)
            assert np.all(err <= HALF[n] * (np.abs(ref) + 32 * U * mag) + 32 * U * mag + TINY[n]), \
                ("q" if k == 0 else "k", float(err.max()))

    def partner(self, z):
        p = np.zeros_like(z)
        r = self.rot
        if r and self.inter:
            p[..., 0:r:2], p[..., 1:r:2] = z[..., 1:r:2], z[..., 0:r:2]
        elif r:
            p[..., :r // 2], p[..., r // 2:r] = z[..., r // 2:r], z[..., :r // 2]
        return p

    def check_bwd(self, out, dw, keep=None):
        cos, sin = self.angles()
        n = _name(self.dt)
        for k in range(2):
            x, w, dy = self.f64(self.x[k]), self.weight(k), self.f64(self.dy[k])
            if x.size == 0:
                continue
            if keep is not None:
                dy = dy * keep[:, :, None, None]
            ref, rw = P.norm_rope_bwd(x, dy, w, self.eps, cos, sin, self.rot, self.inter)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
            dz = np.abs(dy) + self.partner(np.abs(dy))
            gm, xh = dz * np.abs(w), np.abs(x) * r
            mag = r * (gm + xh * (gm * xh).mean(-1, keepdims=True))
            err = np.abs(self.f64(out[k]) - ref)
            assert np.all(err <= HALF[n] * (np.abs(ref) + 64 * U * mag) + 64 * U * mag + TINY[n]), \
                ("dq" if k == 0 else "dk", float(err.max()))
            rows = x.shape[0] * x.shape[1] * x.shape[2]
            ew = np.abs(dw[k].double().cpu().numpy() - rw)
            assert np.all(ew <= (rows + 64) * U * (dz * xh).sum((0, 1, 2)) + 1e-30), float(ew.max())


CASES = [
    # dtype, b, s, h, hk, d, rot, interleaved, weights, positions, layout
    ("bfloat16", 2, 5, 4, 2, 128, 128, False, "16", "random", "bshd"),
    ("float16", 1, 1, 1, 1, 64, 64, False, "32", "index", "bshd"),
    ("float16", 3, 17, 12, 12, 64, 32, True, "16", "random", "bhsd"),
    ("bfloat16", 2, 33, 5, 1, 192, 192, False, "32", "random", "pad"),
    ("float16", 2, 9, 3, 2, 192, 96, False, "16", "index", "bshd"),
    ("bfloat16", 1, 40, 32, 8, 128, 96, False, "none", "random", "pad"),
    ("float16", 2, 7, 9, 3, 128, 16, True, "32", "index", "pad"),
    ("bfloat16", 1, 64, 16, 16, 64, 16, False, "16", "random", "bshd"),
    ("bfloat16", 4, 11, 8, 8, 128, 0, False, "16", "index", "bhsd"),
    ("float16", 1, 130, 17, 5, 192, 192, True, "none", "random", "bhsd"),
    ("float16", 1, 70, 0, 6, 128, 64, False, "16", "random", "bshd"),
    ("bfloat16", 1, 70, 6, 0, 64, 48, True, "16", "random", "bshd"),
    ("bfloat16", 1, 3000, 33, 3, 128, 128, False, "16", "random", "bshd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_parity(case):
    dtype, b, s, h, hk, d, rot, inter, weights, positions, layout = case
    p = Problem(dtype, b, s, h, hk, d, rot, inter, weights, positions, layout, seed=s + d,
                max_pos=max(97, s) if positions == "index" else 97)
    out, ws = p.fwd()
    assert p.ab.attn_query_status(ws) == 0
    p.check_fwd(out)
    out, dw, ws = p.bwd()
    assert p.ab.attn_query_status(ws) == 0
    p.check_bwd(out, dw)
    if layout == "pad":  # what lies between the heads is not written
        base = out[0].permute(0, 2, 1, 3)
        spare = base.as_strided((b, s, h, 8), base.stride(), base.storage_offset() + d)
        assert bool((spare == 7.0).all())


@pytest.mark.parametrize("rot,inter", [(128, False), (32, True), (96, False)])
def test_in_place(rot, inter):
    p = Problem("bfloat16", 2, 37, 6, 2, 128, rot, inter, seed=5)
    want, _ = p.fwd()
    want_b, want_w, _ = p.bwd()
    x = [t.clone() for t in p.x]
    got, _ = p.fwd(out=p.x)
    for a, b in zip(got, want):
        assert p.torch.equal(a, b)
    p.x = x
    got, dw, _ = p.bwd(out=p.dy)
    for a, b in zip(list(got) + dw, want_b + want_w):
        assert p.torch.equal(a, b)


def test_bitwise_reproducible():
    p = Problem("float16", 2, 333, 12, 4, 64, 64, seed=6)
    first = p.bwd()
    for _ in range(3):
        again = p.bwd()
        for a, b in zip(first[0] + first[1], again[0] + again[1]):
            assert p.torch.equal(a, b)


def test_positions_out_of_range_are_flagged_and_zeroed():
    p = Problem("bfloat16", 2, 6, 3, 2, 128, 128, seed=7)
    bad = [(0, 1, -1), (0, 4, 97), (1, 0, 2 ** 31 - 1), (1, 5, -2 ** 31)]
    keep = np.ones((2, 6))
    for n, i, v in bad:
        p.pos[n, i] = v
        keep[n, i] = 0
    out, ws = p.fwd()
    assert p.ab.attn_query_status(ws) == 2
    assert p.ab.attn_query_status(ws) == 0  # read and cleared
    gout, dw, ws = p.bwd()
    assert p.ab.attn_query_status(ws) == 2
    for t in out + gout:
        for n, i, _ in bad:
            assert bool((t[n, :, i] == 0).all())
    for n, i, v in bad:
        p.pos[n, i] = 0
    good, _ = p.fwd()
    m = p.torch.from_numpy(keep).cuda().bool()
    for a, b in zip(out, good):
        assert p.torch.equal(a.permute(0, 2, 1, 3)[m], b.permute(0, 2, 1, 3)[m])
    cos, sin = p.angles()
    for k in range(2):  # they add nothing to the weights' gradients
        _, rw = P.norm_rope_bwd(p.f64(p.x[k]), p.f64(p.dy[k]) * keep[:, :, None, None], p.weight(k), p.eps, cos, sin,
                                p.rot, p.inter)
        r = 1 / np.sqrt((p.f64(p.x[k]) ** 2).mean(-1, keepdims=True) + p.eps)
        dz = np.abs(p.f64(p.dy[k])) + p.partner(np.abs(p.f64(p.dy[k])))
        bound = (2 * 6 * (p.h, p.hk)[k] + 64) * U * (dz * np.abs(p.f64(p.x[k])) * r).sum((0, 1, 2))
        assert np.all(np.abs(dw[k].double().cpu().numpy() - rw) <= bound)


def test_zero_rows_large_rows_and_a_row_with_nan():
    """A zero row gives zeros (eps > 0), a row of the type's largest values stays finite, a row with NaN
    touches no other row."""
    p = Problem("float16", 1, 5, 2, 1, 64, 64, seed=8)
    p.x[0][0, 0, 1] = 0
    p.x[0][0, 1, 2] = 65504
    p.x[1][0, 0, 3, 11] = float("nan")
    out, _ = p.fwd()
    assert bool((out[0][0, 0, 1] == 0).all()) and bool(p.torch.isfinite(out[0]).all())
    assert bool(p.torch.isnan(out[1][0, 0, 3]).all())
    p.x[1][0, 0, 3, 11] = 0
    ref, _ = p.fwd()
    keep = [0, 1, 2, 4]
    assert p.torch.equal(out[1][0, 0, keep], ref[1][0, 0, keep]) and p.torch.equal(out[0], ref[0])


def test_no_tokens():
    p = Problem("bfloat16", 2, 0, 3, 2, 128, 128)
    p.fwd()
    _, dw, ws = p.bwd()
    assert p.ab.attn_query_status(ws) == 0
    assert all(bool((t == 0).all()) for t in dw)


def test_other_stream_and_graph():
    """On a side stream, with a workspace made by the call, and replayed from a graph with new inputs."""
    p = Problem("bfloat16", 2, 200, 8, 2, 128, 128, seed=9)
    torch = p.torch
    want, _ = p.fwd()
    want_b, want_w, _ = p.bwd()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = p.fwd(stream=s)
    got_b, got_w, _ = p.bwd(stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got + got_b + got_w, want + want_b + want_w):
        assert torch.equal(a, b)
    out, gout = [p.new(0), p.new(1)], [p.new(0), p.new(1)]
    dw = [torch.empty(128, device="cuda") for _ in range(2)]
    ws = torch.empty(p.ab.qk_norm_rope_workspace_size(p.desc)[1], dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.fwd(out=out, workspace=ws)
        p.bwd(out=gout, dw=dw, workspace=ws)
    for k in range(2):  # other inputs, then back
        p.x[k].mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    p.check_fwd(out)
    p.check_bwd(gout, dw)


def test_offsets_past_32_bits():
    """Sequences 2.2e9 elements apart."""
    import torch
    p = Problem("bfloat16", 2, 9, 3, 2, 128, 64, seed=10)
    gap = 2_200_000_000
    buf = torch.zeros(gap + 9 * 3 * 128, dtype=p.dt, device="cuda")
    far = buf.as_strided((2, 3, 9, 128), (gap, 128, 3 * 128, 1))
    far.copy_(p.x[0])
    p.x[0] = far
    out, _ = p.fwd()
    p.check_fwd(out)
    want, _ = p.fwd()
    p.fwd(out=[far, out[1]])  # in place
    assert torch.equal(far, want[0])


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 64, False), (64, 32, True), (192, 192, False)])
def test_tokens_out_of_range_beside_values_that_are_not_finite(d, rot, inter):
    """Tokens without a position get zeros, and add nothing to the weights' gradients, whatever their rows, the
    norm weights and the tables hold; row 0 of cos and sin, which no token has, is NaN."""
    p = Problem("bfloat16", 2, 9, 5, 2, d, rot, inter, weights="32", seed=21)
    torch = p.torch
    p.pos.clamp_(min=1)
    for n, i, v in [(0, 0, -1), (0, 5, 97), (1, 8, -7)]:
        p.pos[n, i] = v
    live = (p.pos >= 0) & (p.pos < 97)
    clean, _ = p.fwd()
    clean_b, clean_w, _ = p.bwd()
    p.cos[0] = p.sin[0] = float("nan")
    for t in p.x + p.dy:
        t.permute(0, 2, 1, 3)[~live] = float("nan")
    out, ws = p.fwd()
    assert p.ab.attn_query_status(ws) == 2
    got, dw, _ = p.bwd()
    for a, b in zip(out + got + dw, clean + clean_b + clean_w):
        assert torch.equal(a, b)
    for w in p.w:
        w[3] = float("inf")
        w[d - 1] = float("nan")
    out, _ = p.fwd()
    got, dw, _ = p.bwd()
    for t in out + got:
        assert bool((t.permute(0, 2, 1, 3)[~live] == 0).all())
    for a, b in zip(dw, clean_w):  # the weights' gradients do not depend on the weights
        assert torch.equal(a, b)


def test_status_of_one_call_after_another_on_a_side_stream():
    """Reading a status clears it ahead of the next call on that stream, whose own status is not lost."""
    p = Problem("bfloat16", 1, 6, 2, 1, 64, 64, seed=22)
    torch = p.torch
    p.pos[0, 2] = -1
    s = torch.cuda.Stream()
    out, ws = p.fwd()
    torch.cuda.synchronize()
    for _ in range(200):
        p.fwd(out=out, workspace=ws, stream=s)
        assert p.ab.attn_query_status(ws, s) == 2
    assert p.ab.attn_query_status(ws, s) == 0
