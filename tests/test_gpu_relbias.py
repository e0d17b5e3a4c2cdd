"""GPU parity of sdpa_relbias_fwd_stats / _bwd with the fp64 definition, through the C ABI.

Bounds.  h = eps(type) / 2 is the half step of the 16-bit type, u = 2^-23 covers an fp32 operation (rounded or
truncated).  A score is d exact products summed in fp32, a fused product-sum and a difference, so the exponent
is off by at most (d + 8) u (scale sum|q k| + |bias| + |LSE|), and the exponential adds 2^-21: call the relative
error of P eP.  P and dS are rounded to 16 bits before they are multiplied on (h of the value, and for fp16
2^-25, half its smallest step; in the forward P is relative to a reference at most 2^8 below the row's largest
value).  With A = sum_j P_ij |v_j| and M_ij = P_ij (sum|dO v| + sum|dO O|):
    |O err|  <= h |O| + sum_j (h + 2 max eP + n u) P_ij |v_j| + 2^-25 sum|v|
    |LSE err| <= 2 max_j eP + n u + 2 u |LSE|
    |dS err| <= h |dS| + (eP + (d + 8) u) M + 2^-25;   the gradients are sums of dS (P for dV) times the other
    operand, in fp32 (n u of the sum of magnitudes), rounded once;  dtable sums dS before its rounding.
The factor 2 of the row's largest eP covers the normalisation.  Padding of sequences, the row order of the
sums and the 16-bit outputs' rounding are all within these."""
import numpy as np
import pytest

from oracle import position as P
from tests import harness as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
STEP = {"float16": 2.0 ** -25, "bfloat16": 0.0}


class Problem:
    """lens: [(s_q, s_kv)]; packed when more than one or packed=True.  layout: 'bshd' or 'bhsd'."""

    def __init__(self, dtype, lens, h, hk, d, mask, buckets=32, far=128, both=True, packed=None, b=1, layout="bshd",
                 table="32", seed=0, mode=0, spread=1.5):
        import torch
        import attention_backward_02_gb300 as ab
        self.ab, self.torch = ab, torch
        self.dtype, self.dt = dtype, torch.float16 if dtype == "float16" else torch.bfloat16
        self.packed = len(lens) > 1 if packed is None else packed
        self.lens = list(lens) if self.packed else [lens[0]] * b
        self.h, self.hk, self.d, self.mask, self.far, self.both = h, hk, d, mask, far, both
        self.layout, self.scale = layout, d ** -0.5
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.tq, self.tk = sum(a for a, _ in self.lens), sum(a for _, a in self.lens)
        self.q, self.k, self.v = rnd(self.tq, h, d).to(self.dt), rnd(self.tk, hk, d).to(self.dt), rnd(self.tk, hk, d).to(self.dt)
        self.do = rnd(self.tq, h, d).to(self.dt)
        tt = {"32": torch.float32, "16": self.dt}[table]
        self.table = (rnd(buckets, h) * spread).to(tt).cuda()
        self.bias = ab.relbias(self.table, max_distance=far, bidirectional=both)
        kw = dict(dtype=ab.ATTN_F16 if dtype == "float16" else ab.ATTN_BF16, b=len(self.lens), h=h, h_kv=hk, d=d,
                  scale=self.scale, mask=mask, deterministic=mode)
        if self.packed:
            kw.update(s_q=0, s_kv=0, cu_seqlens_q=list(np.cumsum([a for a, _ in self.lens])),
                      cu_seqlens_kv=list(np.cumsum([a for _, a in self.lens])))
        else:
            kw.update(s_q=lens[0][0], s_kv=lens[0][1])
        self.desc = ab.sdpa_desc(**kw)

    def put(self, t):
        """Token-major [T, n, d] onto the GPU in this problem's layout; returns the tensor that holds it."""
        if self.packed:
            return t.cuda().contiguous()
        b = len(self.lens)
        t = t.cuda().reshape(b, t.shape[0] // b, *t.shape[1:])
        return t.permute(0, 2, 1, 3).contiguous() if self.layout == "bhsd" else t.contiguous()

    def view(self, t):
        if self.packed:
            return self.ab.view_tnd(t)
        return t if self.layout == "bhsd" else t.permute(0, 2, 1, 3)

    def get(self, t):
        """fp64 [T, n, d] of a tensor made by put."""
        if not self.packed:
            t = t.permute(0, 2, 1, 3) if self.layout == "bhsd" else t
            t = t.reshape(-1, *t.shape[2:])
        return t.double().cpu().numpy()

    def nan(self, t):
        return self.put(self.torch.full_like(t, float("nan")))

    def get_lse(self, lse):
        """[T, h] fp64 from the ABI layout."""
        a = lse.double().cpu().numpy()
        if self.packed:
            return a.reshape(self.h, self.tq).T
        b = len(self.lens)
        return a.reshape(b, self.h, -1).transpose(0, 2, 1).reshape(-1, self.h)

    def put_lse(self, a):
        t = self.torch.from_numpy(np.ascontiguousarray(a)).float()
        if self.packed:
            return t.t().contiguous().cuda()
        b = len(self.lens)
        return t.reshape(b, -1, self.h).permute(0, 2, 1).contiguous().cuda()

    def each(self):
        """(query rows, key rows) slices of the sequences."""
        a = c = 0
        for sq, sk in self.lens:
            yield slice(a, a + sq), slice(c, c + sk)
            a, c = a + sq, c + sk

    def f64(self):
        return [x.double().numpy() for x in (self.q, self.k, self.v, self.do)] + [self.table.double().cpu().numpy()]

    def kw(self):
        return dict(scale=self.scale, mask=self.mask, max_distance=self.far, bidirectional=self.both)

    def reference_fwd(self):
        q, k, v, _, t = self.f64()
        o, lse = np.zeros_like(q), np.full(q.shape[:2], np.inf)
        for a, c in self.each():
            o[a], lse[a] = P.relbias_fwd(q[a], k[c], v[c], t, **self.kw())
        return o, lse

    def fwd(self, **kw):
        ten = [self.put(x) for x in (self.q, self.k, self.v)]
        o = self.nan(self.q)
        lse = self.torch.full((self.tq * self.h,), float("nan"), device="cuda")
        ws = self.ab.sdpa_relbias_fwd_stats(self.desc, self.bias, *map(self.view, ten), self.view(o), lse, **kw)
        assert self.ab.attn_query_status(ws, kw.get("stream")) == 0
        return self.get(o), self.get_lse(lse)

    def bwd(self, o, lse, **kw):
        ten = [self.put(x) for x in (self.q, self.k, self.v, o, self.do)]
        out = [self.nan(self.q), self.nan(self.k), self.nan(self.v)]
        dt = self.torch.full(self.table.shape, float("nan"), device="cuda")
        ws = self.ab.sdpa_relbias_bwd(self.desc, self.bias, *map(self.view, ten), self.put_lse(lse),
                                      *map(self.view, out), dt, **kw)
        assert self.ab.attn_query_status(ws, kw.get("stream")) == 0
        return [self.get(x) for x in out] + [dt.double().cpu().numpy()]

    def weights(self, a, c, x, lse):
        """P, its relative error bound and bucket matrix of one sequence and head, from its LSE."""
        q, k, _, _, t = self.f64()
        g = x // (self.h // self.hk)
        sq, sk = q[a].shape[0], k[c].shape[0]
        sh = sk - sq if self.mask == 2 else 0
        bk = P.bucket_matrix(sq, sk, sh, t.shape[0], self.far, self.both)
        s = P._scores(q[a, x], k[c, g], t[:, x], bk, self.scale, self.mask, sh)
        z = np.where(np.isinf(lse), 0.0, lse)[:, None]
        p = np.where(np.isinf(lse)[:, None], 0.0, np.exp(s - z))
        tb = np.where(t[:, x] <= P.MASKED, 0.0, t[:, x])
        ep = (self.d + 8) * U * (self.scale * np.abs(q[a, x]) @ np.abs(k[c, g]).T + np.abs(tb)[bk] + np.abs(z)) + 2.0 ** -21
        return p, ep, bk

    def check_fwd(self, o, lse):
        ro, rl = self.reference_fwd()
        h_, st = HALF[self.dtype], STEP[self.dtype]
        assert np.array_equal(np.isinf(lse), np.isinf(rl)) and not np.isnan(lse).any()
        v = self.f64()[2]
        for a, c in self.each():
            n = c.stop - c.start
            for x in range(self.h):
                p, ep, _ = self.weights(a, c, x, rl[a, x])
                e = ep.max(-1, initial=0.0)
                av = np.abs(v[c, x // (self.h // self.hk)])
                bound = h_ * np.abs(ro[a, x]) + (h_ + 2 * e + n * U)[:, None] * (p @ av) + st * av.sum(0) + 2 * st
                err = np.abs(o[a, x] - ro[a, x])
                assert np.all(err <= bound), ("O", x, float((err - bound).max()))
                live = ~np.isinf(rl[a, x])
                el = np.abs(lse[a, x][live] - rl[a, x][live])
                assert np.all(el <= (2 * e + n * U)[live] + 2 * U * np.abs(rl[a, x][live])), ("LSE", float(el.max()))

    def inputs_bwd(self):
        """O as the type holds it and the fp32 LSE, from the definition."""
        o, lse = self.reference_fwd()
        return self.torch.from_numpy(o).to(self.dt), lse.astype(np.float32)

    def check_bwd(self, got, o, lse):
        q, k, v, do, t = self.f64()
        o, lse = o.double().numpy(), lse.astype(np.float64)
        h_, st = HALF[self.dtype], STEP[self.dtype]
        ref = [np.zeros_like(x) for x in (q, k, v, t)]
        bnd = [np.zeros_like(x) for x in (q, k, v, t)]
        d, sc = self.d, self.scale
        for a, c in self.each():
            r = P.relbias_bwd(q[a], k[c], v[c], o[a], do[a], lse[a], t, **self.kw())
            ref[0][a], ref[1][c], ref[2][c] = r[:3]
            ref[3] += r[3]
            nq, nk = a.stop - a.start, c.stop - c.start
            for x in range(self.h):
                g = x // (self.h // self.hk)
                p, ep, bk = self.weights(a, c, x, lse[a, x])
                ado, av = np.abs(do[a, x]), np.abs(v[c, g])
                ds = np.abs(p * (do[a, x] @ v[c, g].T - (do[a, x] * o[a, x]).sum(-1, keepdims=True)))
                m = p * (ado @ av.T + (ado * np.abs(o[a, x])).sum(-1, keepdims=True))
                e = (ep + (d + 8) * U) * m
                e16 = h_ * ds + e + np.where(p > 0, st, 0.0)
                bnd[0][a, x] += sc * ((e16 + nk * U * ds) @ np.abs(k[c, g]))
                bnd[1][c, g] += sc * ((e16 + nq * self.h * U * ds).T @ np.abs(q[a, x]))
                bnd[2][c, g] += ((h_ + ep + nq * self.h * U) * p + np.where(p > 0, st, 0.0)).T @ ado
                np.add.at(bnd[3][:, x], bk, e + (nq * nk) * 2.0 ** -24 * ds)
        for name, y, r, w in zip(("dQ", "dK", "dV", "dtable"), got, ref, bnd):
            assert np.all(np.isfinite(y)), name
            w = w + (0 if name == "dtable" else h_ * np.abs(r) * (1 + h_) + h_ * w + 2 * st) + 1e-30
            err = np.abs(y - r)
            assert np.all(err <= w), (name, float((err - w).max()), float(err.max()))
        return ref


CASES = [
    # dtype, lens, h, hk, d, mask, buckets, far, both, kw
    ("float16", [(1, 1)], 1, 1, 64, 0, 32, 128, True, {}),
    ("bfloat16", [(128, 128)], 2, 2, 128, 2, 32, 128, False, {}),
    ("float16", [(300, 300)], 4, 2, 64, 0, 32, 128, True, dict(b=2)),
    ("bfloat16", [(257, 511)], 4, 1, 128, 2, 32, 64, True, dict(layout="bhsd")),
    ("float16", [(200, 77)], 2, 1, 64, 2, 16, 100, False, dict(b=2)),          # rows that see no key
    ("bfloat16", [(130, 400)], 2, 2, 64, 1, 64, 256, False, dict(table="16")),
    ("float16", [(640, 640)], 2, 2, 128, 0, 128, 1000, True, dict(table="16", layout="bhsd")),
    ("bfloat16", [(700, 700)], 1, 1, 64, 1, 2, 2, False, {}),                  # the fewest buckets
    ("bfloat16", [(650, 650)], 2, 1, 128, 0, 4, 9, True, {}),                  # far tiles on both sides
    ("float16", [(5, 900)], 3, 3, 128, 2, 32, 128, False, {}),
    ("float16", [(33, 65), (1, 1), (0, 17), (129, 129), (200, 0), (64, 300)], 4, 2, 64, 2, 32, 128, True, {}),
    ("bfloat16", [(127, 127), (385, 384), (3, 250)], 6, 2, 128, 0, 64, 1024, True, {}),
    ("bfloat16", [(140, 300)], 2, 2, 64, 0, 32, 128, True, dict(packed=True)),
    ("bfloat16", [(100, 100)], 2, 2, 128, 2, 32, 65536, False, {}),            # borders past every key
]
ids = lambda c: "-".join(str(x) for x in c).replace(" ", "")


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    p = Problem(*case[:9], seed=len(str(case)), **case[9])
    p.check_fwd(*p.fwd())


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    p = Problem(*case[:9], seed=len(str(case)), **case[9])
    o, lse = p.inputs_bwd()
    p.check_bwd(p.bwd(o, lse), o, lse)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("case", [CASES[2], CASES[3], CASES[10]], ids=ids)
def test_backward_deterministic_modes(case, mode):
    p = Problem(*case[:9], seed=5, mode=mode, **case[9])
    o, lse = p.inputs_bwd()
    first = p.bwd(o, lse)
    p.check_bwd(first, o, lse)
    for a, b in zip(first, p.bwd(o, lse)):
        np.testing.assert_array_equal(a, b)


def test_table_gradient_is_reproducible_with_atomic_dq():
    p = Problem("bfloat16", [(900, 900)], 4, 2, 128, 0, 32, 128, True, seed=6, b=2)
    o, lse = p.inputs_bwd()
    first = p.bwd(o, lse)
    for _ in range(3):
        again = p.bwd(o, lse)
        for i in (1, 2, 3):
            np.testing.assert_array_equal(first[i], again[i])


SHARED = [("bfloat16", [(333, 450)], 8, 2, 128, 2, {}),
          ("float16", [(300, 300)], 12, 4, 64, 0, {}),
          ("bfloat16", [(200, 90), (0, 40), (130, 257)], 6, 2, 128, 1, {}),
          ("float16", [(260, 100)], 8, 1, 64, 2, dict(b=2, layout="bhsd")),
          ("float16", [(90, 500)], 16, 1, 128, 1, {})]


@pytest.mark.parametrize("dtype,lens,h,hk,d,mask,kw", SHARED)
def test_query_heads_of_a_group_in_several_units(dtype, lens, h, hk, d, mask, kw):
    """Few kv heads with many query heads each: dK and dV are sums of fp32 parts, in an order that does not change.
    Rows without keys, keys without queries, lengths of zero and tiles past a sequence's end among them."""
    p = Problem(dtype, lens, h, hk, d, mask, 32, 128, True, seed=14, **kw)
    other = Problem(dtype, lens, h, hk, d, mask, 32, 128, True, seed=14, mode=2, **kw)
    size = [x.ab.sdpa_relbias_workspace_size(x.desc, x.bias)[1] for x in (p, other)]
    assert size[0] - size[1] > 2 * 2 * p.tk * hk * d * 4 - 65536  # (the rule shares these)
    o, lse = p.inputs_bwd()
    first = p.bwd(o, lse)
    p.check_bwd(first, o, lse)
    again = p.bwd(o, lse)
    for i in (1, 2, 3):
        np.testing.assert_array_equal(first[i], again[i])


@pytest.mark.parametrize("dtype,d,mask", [("float16", 64, 2), ("bfloat16", 128, 0)])
def test_masked_buckets(dtype, d, mask):
    """-inf, the type's lowest value and -1e30 mask a bucket; a row left without keys is empty, and nothing of
    it reaches the gradients.  In head 0 everything is masked."""
    p = Problem(dtype, [(150, 150)], 3, 3, d, mask, 8, 20, False, seed=7)
    p.table[0, 1] = -float("inf")
    p.table[7, 1] = p.torch.finfo(p.torch.float32).min
    p.table[3, 2] = -1e30
    p.table[:, 0] = -2e30
    o, lse = p.fwd()
    p.check_fwd(o, lse)
    assert np.all(np.isinf(lse[:, 0])) and np.all(o[:, 0] == 0)
    oi, li = p.inputs_bwd()
    ref = p.check_bwd(p.bwd(oi, li), oi, li)
    assert np.all(ref[3][:, 0] == 0) and ref[3][0, 1] == 0


def test_zero_table_agrees_with_the_plain_call():
    """With a zero table the biased and the plain call are within the bounds of the same definition."""
    import torch
    p = Problem("bfloat16", [(300, 300)], 4, 2, 128, 2, 32, 128, True, seed=8)
    p.table.zero_()
    o, lse = p.fwd()
    p.check_fwd(o, lse)
    ten = [p.put(x) for x in (p.q, p.k, p.v)]
    o2, l2 = p.nan(p.q), torch.empty(p.tq * p.h, device="cuda")
    p.ab.sdpa_fwd_stats(p.desc, *map(p.view, ten), p.view(o2), l2)
    torch.cuda.synchronize()
    p.check_fwd(p.get(o2), p.get_lse(l2))


def test_a_query_with_nan_has_nan_results():
    """Not those of an empty row, and no other row's change."""
    p = Problem("bfloat16", [(140, 140)], 2, 2, 64, 2, 32, 128, True, seed=13)
    o, lse = p.fwd()
    p.q[77, 1, 5] = float("nan")
    o2, lse2 = p.fwd()
    assert np.all(np.isnan(o2[77, 1])) and np.isnan(lse2[77, 1])
    keep = np.ones(o.shape[:2], bool)
    keep[77, 1] = False
    np.testing.assert_array_equal(o[keep], o2[keep])
    np.testing.assert_array_equal(lse[keep], lse2[keep])


def test_no_queries_and_no_keys():
    for lens in [(0, 40), (40, 0), (0, 0)]:
        p = Problem("float16", [lens], 2, 1, 64, 0, 32, 128, True, seed=9)
        o, lse = p.fwd()
        assert np.all(o == 0) and np.all(np.isposinf(lse))
        got = p.bwd(p.torch.from_numpy(o).to(p.dt), lse.astype(np.float32))
        assert all(np.all(x == 0) for x in got)


@pytest.mark.parametrize("d", [64, 128])
def test_plain_backward_without_queries(d):
    """sdpa_bwd with keys that no query sees: zero dK and dV."""
    import torch
    import attention_backward_02_gb300 as ab
    desc = ab.sdpa_desc(dtype=ab.ATTN_F16, b=2, h=4, h_kv=2, s_q=0, s_kv=150, d=d, scale=d ** -0.5)
    k = torch.randn(2, 2, 150, d, device="cuda").half()
    v, none = torch.randn_like(k), torch.empty(2, 4, 0, d, device="cuda", dtype=torch.half)
    dk, dv = torch.full_like(k, float("nan")), torch.full_like(k, float("nan"))
    empty = torch.empty(2, 4, 0, 1, device="cuda")
    ws = torch.empty(max(ab.sdpa_workspace_size(desc)[1], 256), dtype=torch.uint8, device="cuda")
    ab.sdpa_bwd(desc, none, k, v, none, none, empty, none, dk, dv, workspace=ws)
    assert ab.attn_query_status(ws) == 0
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("mode", [1, 2])
def test_graph_replay_and_side_stream(mode):
    """Forward and backward captured with workspaces of their own, replayed with another table and inputs; and
    a direct call on a side stream that makes its own workspace."""
    import torch
    p = Problem("float16", [(260, 300)], 4, 2, 64, 2, 32, 128, True, seed=10, mode=mode)
    ab = p.ab
    q, k, v, do = (p.put(x) for x in (p.q, p.k, p.v, p.do))
    o, lse = p.nan(p.q), torch.empty(p.tq * p.h, device="cuda")
    outs = [p.nan(x) for x in (p.q, p.k, p.v)]
    dt = torch.empty(32, 4, device="cuda")
    wf, wb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in ab.sdpa_relbias_workspace_size(p.desc, p.bias))
    V = p.view

    def both(**kw):
        ab.sdpa_relbias_fwd_stats(p.desc, p.bias, V(q), V(k), V(v), V(o), lse, workspace=kw.get("wf"), stream=kw.get("stream"))
        ab.sdpa_relbias_bwd(p.desc, p.bias, V(q), V(k), V(v), V(o), V(do), lse, *map(V, outs), dt, workspace=kw.get("wb"),
                            stream=kw.get("stream"))

    both(wf=wf, wb=wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(wf=wf, wb=wb)
    p.table.mul_(-0.5)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (o, lse, *outs, dt)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, (o, lse, *outs, dt)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d,h,lens", [
    ("bfloat16", 128, 12, [(1024, 1024)]),                       # units of 256 queries, several a CTA
    ("float16", 64, 20, [(513, 700)]),                           # ... the second 128 past the end
    ("bfloat16", 64, 160, [(200, 130)]),                         # more units than SMs, rows without keys
    ("float16", 128, 40, [(300, 300), (90, 700), (1030, 513), (5, 5), (640, 640)]),  # packed, whole units
])
@pytest.mark.parametrize("mask", [0, 2])
def test_forward_with_many_units(dtype, d, h, lens, mask):
    """Enough units for every CTA to have several, so that what one leaves in shared memory, TMEM and barriers
    meets the next.  The reference takes a few of the heads."""
    p = Problem(dtype, lens, h, h, d, mask, 32, 128, True, seed=h, b=2 if len(lens) == 1 else 1)
    o, lse = p.fwd()
    again, lse2 = p.fwd()
    np.testing.assert_array_equal(o, again)
    np.testing.assert_array_equal(lse, lse2)
    pick = sorted({0, 1, h // 2, h - 1})
    small = Problem(dtype, lens, len(pick), len(pick), d, mask, 32, 128, True, seed=0, b=2 if len(lens) == 1 else 1)
    small.q, small.k, small.v = p.q[:, pick], p.k[:, pick], p.v[:, pick]
    small.table = p.table[:, pick].contiguous()
    small.check_fwd(o[:, pick], lse[:, pick])


def test_two_threads_two_streams():
    """Two threads with a stream, a shape and a workspace each, at once: the results of each alone."""
    import threading
    import torch
    runs, errors = [], []

    def work(p, ten, stream, n):
        ab = p.ab
        q, k, v, do = ten
        outs = []
        for _ in range(n):
            o, lse = torch.empty_like(q), torch.empty(p.tq * p.h, device="cuda")
            g = [torch.empty_like(x) for x in (q, k, v)]
            dt = torch.empty(p.table.shape, device="cuda")
            V = p.view
            ab.sdpa_relbias_fwd_stats(p.desc, p.bias, V(q), V(k), V(v), V(o), lse, stream=stream)
            ab.sdpa_relbias_bwd(p.desc, p.bias, V(q), V(k), V(v), V(o), V(do), lse, *map(V, g), dt, stream=stream)
            outs.append((o, lse, *g, dt))
        return outs

    def guarded(i, *a):
        try:
            runs[i] = work(*a)
        except Exception as e:  # pragma: no cover
            errors.append(e)

    ps = [Problem("float16", [(300, 333)], 4, 2, 64, 2, 32, 128, True, seed=15, mode=2),
          Problem("bfloat16", [(190, 200), (64, 257)], 4, 4, 128, 0, 64, 400, False, seed=16, mode=1)]
    tens = [[p.put(x) for x in (p.q, p.k, p.v, p.do)] for p in ps]
    alone = [work(p, t, None, 1)[0] for p, t in zip(ps, tens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    runs[:] = [None, None]
    threads = [threading.Thread(target=guarded, args=(i, ps[i], tens[i], streams[i], 8)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for want, got in zip(alone, runs):
        for one in got:
            for a, b in zip(want, one):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d,rot", [("bfloat16", 128, 0), ("float16", 64, 32)])
def test_layer(dtype, d, rot):
    """The operators as a layer runs them: norm (and rotation) of the projections, biased attention, and both
    backward, against the fp64 chain.  Each stage's 16-bit result feeds the next, so errors add up: relative
    L2 of 4 half steps per stage, four stages, is the bound for the gradients that went through all of them."""
    import torch
    b, s, h, hk = 2, 190, 4, 2
    p = Problem(dtype, [(s, s)], h, hk, d, 2, 32, 128, False, seed=11, b=b)
    ab = p.ab
    qk = ab.qk_norm_rope_desc(dtype=p.desc.dtype, b=b, s=s, h=h, h_kv=hk, d=d, rotary_dim=rot, max_pos=256 if rot else 0)
    g = torch.Generator().manual_seed(1)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(p.dt).cuda() for _ in range(2)]
    ang = torch.randn(256, max(rot // 2, 1), generator=g)
    cos, sin = (ang.cos().cuda(), ang.sin().cuda()) if rot else (None, None)
    x, y, v, do = (p.put(t) for t in (p.q, p.k, p.v, p.do))
    V = p.view
    q, k, o = torch.empty_like(x), torch.empty_like(y), torch.empty_like(x)
    lse = torch.empty(b, h, s, device="cuda")
    ab.qk_norm_rope_fwd(qk, V(x), V(y), *w, cos, sin, V(q), V(k))
    ab.sdpa_relbias_fwd_stats(p.desc, p.bias, V(q), V(k), V(v), V(o), lse)
    dq, dk, dv, dt = torch.empty_like(x), torch.empty_like(y), torch.empty_like(v), torch.empty_like(p.table)
    ab.sdpa_relbias_bwd(p.desc, p.bias, V(q), V(k), V(v), V(o), V(do), lse, V(dq), V(dk), V(dv), dt)
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    ab.qk_norm_rope_bwd(qk, V(x), V(y), V(dq), V(dk), *w, cos, sin, V(dq), V(dk), *dw)  # in place
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()
    xs = [f(t).reshape(b, s, -1, d) for t in (x, y)]
    c, sn = [(None if t is None else np.broadcast_to(f(t)[:s], (b, s, rot // 2))) for t in (cos, sin)]
    qn, kn = (P.norm_rope(a, f(wi), 1e-6, c, sn, rot, False) for a, wi in zip(xs, w))
    tb, dts, grads = f(p.table), 0, [[], [], []]
    for n in range(b):
        on, ln = P.relbias_fwd(qn[n], kn[n], f(v)[n], tb, **p.kw())
        r = P.relbias_bwd(qn[n], kn[n], f(v)[n], on, f(do)[n], ln, tb, **p.kw())
        dts = dts + r[3]
        for i in range(3):
            grads[i].append(r[i])
    ref = [P.norm_rope_bwd(a, np.stack(gr), f(wi), 1e-6, c, sn, rot, False) for a, gr, wi in zip(xs, grads, w)]
    want = [ref[0][0], ref[1][0], np.stack(grads[2]), dts, ref[0][1], ref[1][1]]
    got = [f(dq), f(dk), f(dv), f(dt), f(dw[0]), f(dw[1])]
    for name, a, r in zip(("dx", "dy", "dv", "dtable", "dwq", "dwk"), got, want):
        a = a.reshape(r.shape)
        assert np.linalg.norm(a - r) <= 16 * HALF[dtype] * np.linalg.norm(r), name


@pytest.mark.parametrize("dtype,d,h,hk", [("float16", 64, 2, 2), ("bfloat16", 128, 4, 2)])
def test_nan_stays_in_its_sequence(dtype, d, h, hk):
    """Infinities and NaN in one packed sequence reach nothing of the others: their outputs and gradients are the
    bits of the clean batch's (dQ in the ordered mode; the table's gradient is shared)."""
    lens = [(70, 100), (45, 61), (130, 150)]
    runs = []
    for bad in (False, True):
        p = Problem(dtype, lens, h, hk, d, 2, 32, 128, True, seed=12, mode=2)
        o, lse = p.inputs_bwd()
        if bad:
            for t, v in ((p.q, float("nan")), (p.do, float("inf")), (o, float("nan"))):
                t[70:115] = v
            for t, v in ((p.k, float("inf")), (p.v, float("nan"))):
                t[100:161] = v
        ten = [p.put(x) for x in (p.q, p.k, p.v)]
        of, lf = p.nan(p.q), p.torch.empty(p.tq * h, device="cuda")
        p.ab.sdpa_relbias_fwd_stats(p.desc, p.bias, *map(p.view, ten), p.view(of), lf)
        runs.append([p.get(of), p.get_lse(lf)] + p.bwd(o, lse)[:3])
    for n, (a, b) in enumerate(zip(*runs)):
        cut = (100, 161) if n in (3, 4) else (70, 115)
        np.testing.assert_array_equal(a[:cut[0]], b[:cut[0]])
        np.testing.assert_array_equal(a[cut[1]:], b[cut[1]:])


def test_table_with_other_memory():
    """The table's tensor given other memory of another type between calls with one bias: as a bias made anew."""
    import torch
    p = Problem("bfloat16", [(150, 170)], 4, 2, 64, 2, 32, 128, True, seed=17)
    o, lse = p.inputs_bwd()
    old = p.table.data
    p.table.data = (torch.randn(32, 4, generator=torch.Generator().manual_seed(3)) * 1.5).bfloat16().cuda()
    old.fill_(float("nan"))
    p.check_fwd(*p.fwd())
    o, lse = p.inputs_bwd()
    p.check_bwd(p.bwd(o, lse), o, lse)
    ab, V = p.ab, p.view
    desc = ab.sdpa_desc(dtype=ab.ATTN_BF16, b=1, h=4, h_kv=2, s_q=1, s_kv=170, d=64, scale=p.scale,
                        mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    q, k, v = (p.put(x) for x in (p.q[:1], p.k, p.v))
    outs = [torch.empty_like(q) for _ in range(2)]
    for bias, out in zip((p.bias, ab.relbias(p.table, max_distance=128)), outs):
        ab.sdpa_relbias_decode(desc, bias, V(q), V(k), V(v), None, V(out))
    assert bool(torch.isfinite(outs[0]).all()) and torch.equal(*outs)


def test_workspace_on_a_side_stream():
    """A workspace made by a call on a side stream is none of the memory that was freed on the current stream, whose
    work on it may still be queued; and it goes back to the side stream."""
    import torch
    p = Problem("float16", [(200, 200)], 4, 2, 64, 2, 32, 128, True, seed=18)
    q, k, v = (p.put(x) for x in (p.q, p.k, p.v))
    o, lse = p.nan(p.q), torch.empty(p.tq * p.h, device="cuda")
    V, s = p.view, torch.cuda.Stream()
    for call, need in ((lambda **kw: p.ab.sdpa_relbias_fwd_stats(p.desc, p.bias, V(q), V(k), V(v), V(o), lse, **kw),
                        p.ab.sdpa_relbias_workspace_size(p.desc, p.bias)[0]),
                       (lambda **kw: p.ab.sdpa_fwd_stats(p.desc, V(q), V(k), V(v), V(o), lse, **kw),
                        max(256, p.ab.sdpa_workspace_size(p.desc)[0]))):
        torch.cuda.synchronize()
        block = torch.empty(need, dtype=torch.uint8, device="cuda")
        freed = block.data_ptr()
        del block
        first = call(stream=s).data_ptr()
        again = call(stream=s).data_ptr()
        own = call().data_ptr()
        torch.cuda.synchronize()
        assert first != freed and again == first and own == freed


@pytest.mark.parametrize("dtype,d,mask,mode", [("float16", 64, 2, 0), ("bfloat16", 128, 0, 2), ("bfloat16", 64, 1, 1)])
def test_rows_behind_the_last_sequence(dtype, d, mask, mode):
    """Packed tensors with more rows than the sequences have: those of the inputs (NaN here) are not looked at, those of
    the outputs stay as they were."""
    import torch
    lens, h, hk = [(70, 100), (45, 61), (130, 150)], 4, 2
    p = Problem(dtype, lens, h, hk, d, mask, 32, 128, True, seed=19, mode=mode)
    o, lse = p.inputs_bwd()
    ab, V = p.ab, p.view
    longer = lambda t: torch.cat([t, torch.full((133, *t.shape[1:]), float("nan"), dtype=t.dtype)]).cuda()
    q, k, v, do, oin = (longer(t) for t in (p.q, p.k, p.v, p.do, o))
    out = [torch.full_like(t, 3.0) for t in (q, q, k, v)]
    l2, dt = torch.full((h * p.tq,), float("nan"), device="cuda"), torch.empty_like(p.table)
    ab.sdpa_relbias_fwd_stats(p.desc, p.bias, V(q), V(k), V(v), V(out[0]), l2)
    ws = ab.sdpa_relbias_bwd(p.desc, p.bias, V(q), V(k), V(v), V(oin), V(do), p.put_lse(lse), *map(V, out[1:]), dt)
    assert ab.attn_query_status(ws) == 0
    for t, n in zip(out, (p.tq, p.tq, p.tk, p.tk)):
        assert bool((t[n:] == 3.0).all())
    p.check_fwd(p.get(out[0][:p.tq]), p.get_lse(l2))
    p.check_bwd([p.get(t[:n]) for t, n in zip(out[1:], (p.tq, p.tk, p.tk))] + [dt.double().cpu().numpy()], o, lse)
