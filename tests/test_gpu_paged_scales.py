"""Scales of an e4m3 cache that its caller made: of either sign, and far from one another.  A value's scale may only matter
as far as its key's weight does.

Bounds (u = 2^-23, g = 2^-11, half a step of the half-precision type): a key's score is off by at most
e = (d + 8) u (sum |q k| scale + |s|) + 2 u |s - largest s| + 4 u (|E| + largest |E|), E the exponents of the value scales
(they are added to the scores where the weights are taken); its weight is rounded to half precision, which is off by
g of it or by 2^-25 of the largest weight times scale that the row sees, E rounding that up by less than 2; its value may be a
number times the scale's fraction, both rounded (2 g):
    |O err| <= h |O| + sum_j (3 g + e_j + sum P e + 2^-20 + n u) P_j |v_j| + 2^-24 max_j (P_j |scale_j|) sum_j |code_j|
    |LSE err| <= sum P e + 2^-20 + n u + 4 u (|LSE| + largest |E|)
over the keys j that the row sees (h: half a step of the output's type; fp16 outputs are off by 2^-25 at least)."""
import numpy as np
import pytest

from oracle import paged as P
from tests.paged_problem import HALF, U, Problem

pytestmark = pytest.mark.gpu

# new tokens, query heads: 8 and 16 rows of the mma.sync kernel, 128 and 256 of the tensor-core kernel
FORMS = [(1, 4), (5, 4), (30, 4), (150, 4)]


def _set(p, side, scales):
    """The cache's key (0) or value (1) scales: scales [slot, head] where a sequence has a token."""
    import torch
    live = ~p.scales[side].isnan()
    p.scales[side][live] = torch.as_tensor(scales, dtype=torch.float32).reshape(p.scales[side].shape)[live]
    p.cscales[side].copy_(p.scales[side])


def _slot_scales(p, side):
    return p.scales[side].reshape(-1, p.hk).numpy().copy()


def _check(p, o, lse):
    o = p.packed_of(o).double().cpu().numpy()
    lse = lse.double().cpu().numpy() if p.packed else lse.permute(1, 0, 2).reshape(p.h, -1).double().cpu().numpy()
    grp, g, h = p.h // p.hk, 2.0 ** -11, HALF[p.dtype]
    for n, m in enumerate(p.new):
        k, v = p.contents(n)
        rows = slice(p.starts[n], p.starts[n] + m)
        size = np.repeat(np.abs(p.scales[1].reshape(-1, p.hk)[p.rows_of[n]].double().numpy()), grp, 1).T  # [h, n]
        code = np.repeat(np.abs(P.E4M3[p.pool[1].reshape(-1, p.hk, p.d)[p.rows_of[n]].numpy()]), grp, 1)
        ref, rl, w, mag, s = P.attention(p.q[rows].double().numpy(), k, v, p.scale, p.causal)
        seen = np.arange(len(k))[None, :] <= (np.arange(m) + len(k) - m)[:, None] if p.causal else np.ones((m, len(k)), bool)
        seen = seen[:, None, :]
        top = np.where(seen, s, -np.inf).max(-1, keepdims=True)
        exps = np.abs(np.log2(np.clip(size, 2.0 ** -80, None)))
        most = np.where(seen, exps, 0).max(-1, initial=0, keepdims=True)
        e = np.where(seen, (p.d + 8) * U * (mag + np.abs(s)) + 2 * U * np.abs(s - top) + 4 * U * (exps + most), 0)
        pe = (w * e).sum(-1, keepdims=True)
        av = np.repeat(np.abs(v), grp, 1)
        small = 2.0 ** -24 * (w * size).max(-1)[..., None] * np.einsum("mhn,nhd->mhd", np.where(seen, 1.0, 0.0) + 0 * w, code)
        bound = (h * np.abs(ref) + np.einsum("mhn,nhd->mhd", (3 * g + e + pe + 2.0 ** -20 + len(k) * U) * w, av) + small +
                 (2.0 ** -25 if p.dtype == "float16" else 2.0 ** -126))
        err = np.abs(o[rows] - ref)
        assert np.all(err <= bound), (n, float(np.nanmax(err)), float(np.nanmax(err / bound)), int(np.isnan(err).sum()))
        lim = pe[..., 0] + 2.0 ** -20 + len(k) * U + 4 * U * (np.abs(rl) + most[..., 0])
        err = np.abs(lse[:, rows].T - rl)
        assert np.all(err <= lim), (n, float(np.nanmax(err)), float(np.nanmax(err / lim)))
    return ref


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,h", FORMS)
@pytest.mark.parametrize("signs", ["all", "mixed"])
def test_scales_below_zero(dtype, d, new, h, signs):
    """A row stands for code * scale whatever the scale's sign."""
    import torch
    p = Problem(dtype, "e4m3", [300, 170], [new, new], h, 1, d, packed=False, seed=21)
    rng = np.random.default_rng(22)
    for side in range(2):
        x = _slot_scales(p, side)
        sign = -1.0 if signs == "all" else rng.choice([-1.0, 1.0], x.shape)
        _set(p, side, x * sign * (2.0 ** rng.integers(-3, 4, x.shape) if side else 1.0))
    o, lse = p.attend()
    _check(p, o, lse)
    back = [torch.empty(2, 1, new, d, dtype=p.dt, device="cuda") for _ in range(2)]
    p.ab.paged_cache_read(p.desc, p.cache, p.dtable, p.dlens, *back)
    for n in range(2):
        for side in range(2):
            want = p.contents(n)[side][-new:]
            assert np.all(np.abs(back[side][n, 0].double().cpu().numpy() - want[:, 0]) <= HALF[dtype] * np.abs(want[:, 0]) + 2.0 ** -25)


def _light_key(p, n, key, head=0):
    """Puts a cached key where every query's score is about -45: element 0 of the queries is 4, of the key the rest."""
    import torch
    slot = p.rows_of[n][key]
    code, size = P.quantise(np.array([[-45.0 / (4 * p.scale)] + [0.0] * (p.d - 1)], np.float32))
    p.pool[0].reshape(-1, p.hk, p.d)[slot, head] = torch.from_numpy(code[0])
    p.scales[0].reshape(-1, p.hk)[slot, head] = float(size[0])
    p.cpool[0].view(torch.uint8).copy_(p.pool[0])
    p.cscales[0].copy_(p.scales[0])


@pytest.mark.parametrize("dtype,up", [("bfloat16", 22), ("bfloat16", 40), ("float16", 20)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,h", FORMS)
@pytest.mark.parametrize("where", [3, 70, 200])
def test_a_large_value_of_negligible_weight(dtype, up, d, new, h, where):
    """One key of a weight of about 2^-65 whose value's scale is 2^20 to 2^40 above the rest: 2^-25 of them at most."""
    p = Problem(dtype, "e4m3", [400], [new], h, 1, d, packed=False, seed=23)
    p.q[..., 0] = 4
    _light_key(p, 0, where)
    x = _slot_scales(p, 1) * (2.0 ** -8 if dtype == "float16" else 1.0)  # (its value within the type's range)
    x[p.rows_of[0][where]] = np.nanmedian(x) * 2.0 ** up
    _set(p, 1, x)
    o, lse = p.attend()
    _check(p, o, lse)


@pytest.mark.parametrize("dtype,up", [("bfloat16", 22), ("bfloat16", 60), ("float16", 20)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,h", [f for f in FORMS if f[0] > 1])
def test_a_large_value_that_earlier_tokens_do_not_see(dtype, up, d, new, h):
    """The last token's value is 2^20 to 2^60 above the rest: the rows before it do not see it, and their outputs are
    those of a cache without it."""
    import torch
    outs = []
    for raised in (False, True):
        p = Problem(dtype, "e4m3", [300, 128 + new], [new, new], h, 1, d, packed=False, seed=24)
        x = _slot_scales(p, 1) * (2.0 ** -8 if dtype == "float16" else 1.0)
        if raised:
            for n in range(2):
                x[p.rows_of[n][-1]] = np.nanmedian(x) * 2.0 ** up
        _set(p, 1, x)
        o, lse = p.attend()
        _check(p, o, lse)
        outs.append(o[:, :, :-1])
    assert torch.equal(*outs)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,h", FORMS)
def test_dominant_keys_of_small_scales(d, new, h):
    """Value scales from 2^-30 to 2^30, larger the lighter their key: weight times scale is about the same for all."""
    p = Problem("bfloat16", "e4m3", [500], [new], h, 1, d, packed=False, seed=25)
    p.q[:] = p.q[:1, :1]  # (one query for all rows, so that its weights are known)
    k, _ = p.contents(0)
    s = (k[:, 0] @ p.q[0, 0].double().numpy()) * p.scale
    x = _slot_scales(p, 1)
    x[p.rows_of[0], 0] = np.clip(np.exp(-(s - s.mean()) * 3), 2.0 ** -30, 2.0 ** 30)
    p.causal, p.desc.mask = False, p.ab.ATTN_MASK_NONE
    _set(p, 1, x)
    o, lse = p.attend()
    _check(p, o, lse)


@pytest.mark.parametrize("new,h", FORMS)
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -118, 2.0 ** -70, 2.0 ** 70])
def test_scales_alike_and_far_from_one(new, h, scale):
    """A sequence whose value scales are all zero or the least there is (rows of zeros), or all small or large."""
    p = Problem("bfloat16", "e4m3", [700, 33], [min(new, 33)] * 2, h, 1, 128, packed=False, seed=26)
    x = np.full_like(_slot_scales(p, 1), scale)
    _set(p, 1, x)
    o, lse = p.attend()
    if scale in (0.0, 2.0 ** -118):  # (values below 2^-109: their outputs are what is left of them)
        assert bool((o.abs() <= 2.0 ** -100).all())
        o = o * 0
        p.scales[1][~p.scales[1].isnan()] = 0
    _check(p, o, lse)


@pytest.mark.parametrize("new,h", FORMS)
def test_one_scale_for_all_rows(new, h):
    """Scales of stride 0, as expand makes them, are read through: the bits of the same calls on copies.  A write is refused."""
    import torch
    outs = []
    for copies in (False, True):
        p = Problem("bfloat16", "e4m3", [300, 170], [new, new], h, 1, 128, packed=False, seed=27)
        size = [torch.full((1, 1, 1), x, device="cuda").expand(p.cscales[0].shape) for x in (0.011, 0.0075)]
        if copies:
            size = [t.contiguous() for t in size]
        cache = p.ab.paged_cache(*p.cpool, k_scale=size[0], v_scale=size[1])
        p.cache = cache
        o, lse = p.attend()
        back = [torch.empty(2, 1, new, 128, dtype=p.dt, device="cuda") for _ in range(2)]
        p.ab.paged_cache_read(p.desc, cache, p.dtable, p.dlens, *back)
        outs.append([o, lse, *back])
        if not copies:
            with pytest.raises(p.ab.AttnError):
                p.ab.paged_cache_write(p.desc, cache, p.dtable, p.dlens, *back)
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*outs))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,h", [(1, 4), (5, 4), (30, 4), (70, 4)])
def test_scales_far_apart_over_many_pieces(d, new, h):
    """A long sequence, whose pieces several blocks hold and join: one key in a hundred has a value scale up to 2^30 above or
    below the others, of either sign, one in a hundred has a scale of zero."""
    p = Problem("bfloat16", "e4m3", [9000, 77], [new, new], h, 1, d, packed=False, page=64, seed=28)
    rng = np.random.default_rng(29)
    x = _slot_scales(p, 1)
    at = rng.random(x.shape)
    x = np.where(at < 0.01, x * 2.0 ** rng.integers(-30, 31, x.shape) * rng.choice([-1.0, 1.0], x.shape), x)
    x = np.where(at > 0.99, 0.0 * x, x)
    _set(p, 1, x)
    o, lse = p.attend()
    _check(p, o, lse)


@pytest.mark.parametrize("new,h", FORMS)
def test_a_bad_page_of_an_e4m3_cache_reads_as_zeros(new, h):
    """Its keys have the score 0 and its values are zeros, and the call says so."""
    p = Problem("bfloat16", "e4m3", [400, 300], [new, new], h, 1, 128, packed=False, seed=30)
    for n, i in ((0, 2), (1, 0)):
        p.dtable[n, i] = -3
        slots = p.rows_of[n][16 * i:16 * i + 16]
        for side in range(2):
            p.pool[side].reshape(-1, 1, 128)[slots] = 0
            p.scales[side].reshape(-1, 1)[slots] = 0
    o, lse = p.attend(flags=2)
    _check(p, o, lse)
