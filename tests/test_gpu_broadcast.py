"""Inputs that are one and the same for all sequences, heads or tokens (a stride of 0, as expand makes them): every
fixed-length call gives the bits of the same call on copies."""
import pytest

pytestmark = pytest.mark.gpu

# (dimension of [b, heads, tokens, d] that q, k, v, o, dO repeat along; None: none)
REPEATS = [(None, 0, 0, None, 0), (0, 1, 1, 0, 1), (1, 2, 0, 1, 2), (2, 0, 2, 2, 0), (0, None, None, 0, None)]


def _inputs(dtype, b, h, hk, s_q, s_kv, d, repeats, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, (heads, s) in enumerate([(h, s_q), (hk, s_kv), (hk, s_kv), (h, s_q), (h, s_q)]):
        shape = [b, heads, s, d]
        base = list(shape)
        if repeats[n] is not None:
            base[repeats[n]] = 1
        out.append(torch.randn(*base, generator=g).to(getattr(torch, dtype)).cuda().expand(*shape))
    return out


@pytest.mark.parametrize("dtype,d,h,hk", [("float16", 64, 4, 2), ("bfloat16", 128, 6, 3)])
@pytest.mark.parametrize("repeats", REPEATS, ids=str)
@pytest.mark.parametrize("biased", [False, True])
def test_attention(dtype, d, h, hk, repeats, biased):
    import torch
    import attention_backward_02_gb300 as ab
    b, s_q, s_kv = 3, 150, 213
    desc = ab.sdpa_desc(dtype=ab.ATTN_F16 if dtype == "float16" else ab.ATTN_BF16, b=b, h=h, h_kv=hk, s_q=s_q, s_kv=s_kv,
                        d=d, scale=d ** -0.5, mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT, deterministic=ab.ATTN_DQ_ORDERED)
    table = torch.randn(32, h, generator=torch.Generator().manual_seed(1)).cuda()
    bias = ab.relbias(table)
    runs = []
    for copies in (False, True):
        given = _inputs(dtype, b, h, hk, s_q, s_kv, d, repeats, seed=d)
        q, k, v, o_in, do = [t.contiguous() for t in given] if copies else given
        new = lambda n, s: torch.full((b, n, s, d), float("nan"), dtype=q.dtype, device="cuda")
        o, lse = new(h, s_q), torch.full((b, h, s_q), float("nan"), device="cuda")
        grads = [new(h, s_q), new(hk, s_kv), new(hk, s_kv)]
        if biased:
            dt = torch.full_like(table, float("nan"))
            wf = ab.sdpa_relbias_fwd_stats(desc, bias, q, k, v, o, lse)
            wb = ab.sdpa_relbias_bwd(desc, bias, q, k, v, o_in, do, lse, *grads, dt)
            grads.append(dt)
        else:
            wf = ab.sdpa_fwd_stats(desc, q, k, v, o, lse)
            wb = ab.sdpa_bwd(desc, q, k, v, o_in, do, lse, *grads)
        assert ab.attn_query_status(wf) == 0 and ab.attn_query_status(wb) == 0
        runs.append([o, lse, *grads])
    for n, (x, y) in enumerate(zip(*runs)):
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y), n


@pytest.mark.parametrize("repeats", REPEATS, ids=str)
def test_decode_and_norm(repeats):
    import torch
    import attention_backward_02_gb300 as ab
    b, h, hk, s, d = 3, 6, 3, 213, 128
    q, k, v, x, dy = _inputs("bfloat16", b, h, hk, 1, s, d, repeats, seed=5)
    desc = ab.sdpa_desc(dtype=ab.ATTN_BF16, b=b, h=h, h_kv=hk, s_q=1, s_kv=s, d=d, scale=d ** -0.5,
                        mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    bias = ab.relbias(torch.randn(32, h, generator=torch.Generator().manual_seed(1)).cuda())
    lens = torch.tensor([213, 7, 100], dtype=torch.int32, device="cuda")
    norm = ab.qk_norm_rope_desc(dtype=ab.ATTN_BF16, b=b, s=1, h=h, h_kv=0, d=d)
    runs = []
    for c in (lambda t: t, lambda t: t.contiguous()):
        o, y, dx = (torch.empty(b, h, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        dw = torch.empty(d, device="cuda")
        ab.sdpa_relbias_decode(desc, bias, c(q), c(k), c(v), lens, o)
        ab.qk_norm_rope_fwd(norm, c(x), None, None, None, None, None, y, None)
        ab.qk_norm_rope_bwd(norm, c(x), None, c(dy), None, None, None, None, None, dx, None, dw)
        runs.append([o, y, dx, dw])
    for a, e in zip(*runs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, e)
