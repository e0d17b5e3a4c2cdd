"""GPU parity of sdpa_relbias_decode with the fp64 definition.

Bounds as in the forward's (h half step of the 16-bit type, u = 2^-23): the exponent of a key's weight is off by
at most (d + 8) u (scale sum|q k| + |bias| + |s max|), the exponential by 2^-21, together eP; weights are
rounded to 16 bits (h, and for fp16 2^-25 relative to the largest) before the product with V:
    |O err| <= h |O| + sum_j (h + 2 max eP + n u) P_j |v_j| + 2^-25 sum|v| + half the smallest step."""
import numpy as np
import pytest

from oracle import position as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
STEP = {"float16": 2.0 ** -25, "bfloat16": 0.0}


class Problem:
    def __init__(self, dtype, lens, cap, h, hk, d, buckets=32, far=128, both=False, layout="bshd", seed=0, table="32"):
        import torch
        import attention_backward_02_gb300 as ab
        self.ab, self.torch, self.dtype = ab, torch, dtype
        self.dt = torch.float16 if dtype == "float16" else torch.bfloat16
        self.lens, self.cap, self.h, self.hk, self.d, self.far, self.both = list(lens), cap, h, hk, d, far, both
        b = len(self.lens)
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn(b, h, 1, d, generator=g).to(self.dt).cuda()
        kv = [torch.randn(b, hk, cap, d, generator=g).to(self.dt) for _ in range(2)]
        for n, c in enumerate(self.lens):  # what lies behind the cached keys must not be looked at
            for t in kv:
                t[n, :, min(max(c, 0), cap):] = float("nan")
        if layout == "bshd":
            kv = [t.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for t in kv]
        elif layout == "kv":  # keys and values of a token side by side
            both_ = torch.stack([t.permute(0, 2, 1, 3) for t in kv], 3).contiguous().cuda()
            kv = [both_[:, :, :, i].permute(0, 2, 1, 3) for i in range(2)]
        else:
            kv = [t.cuda() for t in kv]
        self.k, self.v = kv
        self.table = (torch.randn(buckets, h, generator=g) * 1.5).to({"32": torch.float32, "16": self.dt}[table]).cuda()
        self.bias = ab.relbias(self.table, max_distance=far, bidirectional=both)
        self.desc = ab.sdpa_desc(dtype=ab.ATTN_F16 if dtype == "float16" else ab.ATTN_BF16, b=b, h=h, h_kv=hk, s_q=1,
                                 s_kv=cap, d=d, scale=d ** -0.5, mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def run(self, flags=0, use_lens=True, **kw):
        o = self.torch.full_like(self.q, float("nan"))
        ws = self.ab.sdpa_relbias_decode(self.desc, self.bias, self.q, self.k, self.v, self.dlens if use_lens else None, o,
                                         **kw)
        assert self.ab.attn_query_status(ws, kw.get("stream")) == flags
        return o

    def check(self, o, lens=None):
        o, q, t = (x.double().cpu().numpy() for x in (o, self.q, self.table))
        k, v = (x.double().cpu().numpy() for x in (self.k, self.v))
        for n, c in enumerate(self.lens if lens is None else lens):
            c = min(max(c, 0), self.cap)
            kk, vv = k[n, :, :c].transpose(1, 0, 2), v[n, :, :c].transpose(1, 0, 2)
            ref, lse = P.relbias_fwd(q[n].transpose(1, 0, 2), kk, vv, t, self.d ** -0.5, 2, self.far, self.both)
            bk = P.bucket_matrix(1, c, c - 1, t.shape[0], self.far, self.both)[0] if c else np.zeros(0, int)
            for x in range(self.h):
                g = x // (self.h // self.hk)
                if np.isinf(lse[0, x]):
                    assert np.all(o[n, x, 0] == 0)
                    continue
                s = P._scores(q[n, x], kk[:, g], t[:, x], bk[None], self.d ** -0.5, 2, c - 1)[0]
                p = np.exp(s - lse[0, x])
                tb = np.where(t[:, x] <= P.MASKED, 0, t[:, x])[bk]
                e = ((self.d + 8) * U * (self.d ** -0.5 * np.abs(kk[:, g]) @ np.abs(q[n, x, 0]) + np.abs(tb) +
                                         np.abs(s[s > -np.inf]).max()) + 2.0 ** -21).max()
                h_, st = HALF[self.dtype], STEP[self.dtype]
                av = np.abs(vv[:, g])
                bound = h_ * np.abs(ref[0, x]) + (h_ + 2 * e + c * U) * (p @ av) + st * av.sum(0) + 2 * st
                err = np.abs(o[n, x, 0] - ref[0, x])
                assert np.all(err <= bound), (n, x, c, float(err.max()), float((err - bound).max()))


CASES = [
    # dtype, lens, cap, h, hk, d, kw
    ("float16", [1], 1, 1, 1, 64, {}),
    ("bfloat16", [1, 2, 15, 16, 17, 63, 64, 65, 0], 70, 4, 2, 128, {}),
    ("float16", [1000], 1024, 12, 12, 64, {}),
    ("bfloat16", [1, 700, 333, 2000], 2000, 8, 1, 128, dict(layout="kv", table="16")),
    ("float16", [129, 640, 90], 640, 32, 2, 128, dict(layout="bhsd")),       # 16 query heads a group
    ("bfloat16", [300, 5], 301, 35, 1, 64, dict(both=True, buckets=64, far=1000)),  # 35 a group: three row blocks
    ("float16", [5000, 4097], 5000, 9, 1, 64, dict(buckets=16, far=40)),
    ("bfloat16", [2500] * 3, 2600, 6, 2, 128, dict(buckets=2, far=2)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_parity(case):
    p = Problem(*case[:6], seed=case[2], **case[6])
    o = p.run()
    p.check(o)
    assert p.torch.equal(o, p.run())  # bitwise reproducible


def test_whole_cache_without_lengths():
    p = Problem("bfloat16", [400, 400], 400, 4, 4, 128, seed=1)
    assert p.torch.equal(p.run(), p.run(use_lens=False))


def test_lengths_out_of_range_are_flagged_and_brought_in():
    p = Problem("float16", [-3, 90, 50, 2 ** 31 - 1], 80, 4, 2, 64, seed=2)
    p.check(p.run(flags=2))
    p = Problem("float16", [0, 0], 3000, 4, 2, 64, seed=2)
    assert bool((p.run() == 0).all())


@pytest.mark.parametrize("cap", [48, 900])
def test_masked_buckets(cap):
    p = Problem("bfloat16", [40, 30], cap, 3, 1, 128, 32, 128, seed=3)
    p.table[:, 0] = -float("inf")       # nothing left: O = 0
    p.table[5:, 1] = -3e38              # the last five keys
    o = p.run()
    p.check(o)
    assert bool((o[:, 0] == 0).all()) and bool(p.torch.isfinite(o).all())


def test_graph_follows_a_growing_cache():
    """One captured step, replayed as the cache grows: the norm writes the new token's key into its place of the
    cache (a strided view), then the token attends to everything cached."""
    import torch
    p = Problem("bfloat16", [0, 0], 300, 4, 2, 128, seed=4)
    ab, cap = p.ab, 300
    g = torch.Generator().manual_seed(5)
    raw_k, raw_v = (torch.randn(2, 2, cap, 128, generator=g).to(p.dt).cuda() for _ in range(2))
    p.k.zero_(); p.v.zero_()
    qd = ab.qk_norm_rope_desc(dtype=p.desc.dtype, b=2, s=1, h=0, h_kv=2, d=128)
    ws = torch.empty(ab.sdpa_relbias_decode_workspace_size(p.desc, p.bias), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(p.q)
    ab.sdpa_relbias_decode(p.desc, p.bias, p.q, p.k, p.v, p.dlens, o, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ab.sdpa_relbias_decode(p.desc, p.bias, p.q, p.k, p.v, p.dlens, o, workspace=ws)
    for n in range(cap):
        ab.qk_norm_rope_fwd(qd, None, raw_k[:, :, n:n + 1], None, None, None, None, None, p.k[:, :, n:n + 1])
        p.v[:, :, n] = raw_v[:, :, n]
        p.dlens.fill_(n + 1)
        graph.replay()
        if n in (0, 1, 63, 64, 200, 299):
            torch.cuda.synchronize()
            p.check(o, [n + 1, n + 1])
    x = raw_k.double()
    want = x / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt()
    assert bool(((p.k.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all())


def test_the_training_forward_agrees():
    """The last row of the biased forward and the decode step are the same attention."""
    import torch
    p = Problem("float16", [257, 257], 257, 6, 2, 64, seed=6)
    desc = p.ab.sdpa_desc(dtype=p.desc.dtype, b=2, h=6, h_kv=2, s_q=1, s_kv=257, d=64, scale=64 ** -0.5,
                          mask=p.ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    o, lse = torch.empty_like(p.q), torch.empty(2, 6, 1, device="cuda")
    p.ab.sdpa_relbias_fwd_stats(desc, p.bias, p.q, p.k, p.v, o, lse)
    p.check(o)
    p.check(p.run())


def test_offsets_past_32_bits():
    """A cache of 2.3e9 elements: the last sequence's keys lie beyond 2^31 elements.  First a few of its keys, then
    a length that spans all of it: zeros but for the last 64 keys.  (Bound there: the P rounding 2^-8 of the
    magnitude and of the output, and half of it again for 380000 fp32 terms of equal sign.)"""
    import torch
    import attention_backward_02_gb300 as ab
    b, cap, h, d = 3, 380000, 16, 128
    p = Problem("bfloat16", [0, 0, 64], 64, h, h, d, seed=8)
    big = [torch.zeros(b, cap, h, d, dtype=p.dt, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31
    for t, x in zip(big, (p.k, p.v)):
        t[2, :64] = x[2].permute(1, 0, 2)
    k, v = (t.permute(0, 2, 1, 3) for t in big)
    desc = ab.sdpa_desc(dtype=p.desc.dtype, b=b, h=h, h_kv=h, s_q=1, s_kv=cap, d=d, scale=d ** -0.5,
                        mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    o = torch.full_like(p.q, float("nan"))
    ws = ab.sdpa_relbias_decode(desc, p.bias, p.q, k, v, p.dlens, o)
    assert ab.attn_query_status(ws) == 0
    p.check(o)
    p.dlens[2] = cap
    for t, x in zip(big, (p.k, p.v)):
        t[2, :64] = 0
        t[2, cap - 64:] = x[2].permute(1, 0, 2)
    ab.sdpa_relbias_decode(desc, p.bias, p.q, k, v, p.dlens, o)
    table = p.table.double()
    bucket = torch.full((cap,), 31, device="cuda")
    bucket[cap - 200:] = torch.tensor([P.bucket(x, 32, 128, False) for x in range(-199, 1)], device="cuda")
    want, mag = torch.empty(h, d, device="cuda", dtype=torch.float64), torch.empty(h, d, device="cuda", dtype=torch.float64)
    for x in range(h):
        kk, vv = big[0][2, :, x].double(), big[1][2, :, x].double()
        w = torch.softmax(kk @ p.q[2, x, 0].double() * d ** -0.5 + table[bucket, x], -1)
        want[x], mag[x] = w @ vv, w @ vv.abs()
    bound = 2.0 ** -8 * (want.abs() + 1.5 * mag) + 1e-6
    assert bool(((o[2, :, 0].double() - want).abs() <= bound).all())
