"""The norm weights' gradients where every term dz xh is positive, so that rows which are lost or counted twice show:
with random signs they may hide behind the rounding that a bound has to allow.

Inputs and gradients are positive and the angles small, so that dz = Rot^T dy is positive too.  Bounds (u = 2^-24): a
term is off by at most 24 u (|dy_a| + |dy_b|) xh, as in the norm's tests.  It passes an addition for each item (four
heads of a token) of its warp, 2 between the lanes that hold a row each, 4 over the warps of a block, one for every 32nd
block and 5 between lanes, each off by at most u of a sum of positive terms.  The fewest blocks a side can have with
enough work are its share of two an SM."""
import math

import numpy as np
import pytest

from oracle import position as P

U = 2.0 ** -24
SMS, MOST_BLOCKS = 152, 1216

CASES = [
    # dtype, b, s, h, hk, d, rot, interleaved
    ("bfloat16", 1, 3000, 33, 3, 128, 128, False),
    ("float16", 2, 901, 12, 12, 64, 32, True),
    ("bfloat16", 1, 1777, 16, 1, 192, 64, False),
    ("float16", 3, 500, 5, 5, 128, 0, False),
]


def inputs(case):
    """x, dy (each of q and k) [b, s, n, d] CPU tensors of the type; cos, sin fp32 [97, rot / 2]; positions [b, s]."""
    import torch
    dtype, b, s, h, hk, d, rot, _ = case
    dt, g = getattr(torch, dtype), torch.Generator().manual_seed(s + d)
    some = lambda *n: torch.rand(*n, generator=g)
    x = [(0.5 + some(b, s, n, d)).to(dt) for n in (h, hk)]
    dy = [(1 + some(b, s, n, d)).to(dt) for n in (h, hk)]
    ang = some(97, max(rot // 2, 1)) * 0.2
    return x, dy, ang.cos(), ang.sin(), torch.randint(0, 97, (b, s), generator=g, dtype=torch.int32)


def terms(case, x, dy, cos, sin, pos):
    """dz xh and its error bound, fp64 [b, s, n, d]."""
    *_, d, rot, inter = case
    x, dy, rows = x.double().numpy(), dy.double().numpy(), pos.numpy()
    c, sn = cos.double().numpy()[rows], sin.double().numpy()[rows]
    xh = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
    other = np.zeros_like(dy)
    if rot and inter:
        other[..., 0:rot:2], other[..., 1:rot:2] = dy[..., 1:rot:2], dy[..., 0:rot:2]
    elif rot:
        other[..., :rot // 2], other[..., rot // 2:rot] = dy[..., rot // 2:rot], dy[..., :rot // 2]
    dz = P._turn(dy, c, -sn, rot, inter)
    assert np.all(dz > 0)
    return dz * xh, 24 * U * (dy + other) * xh


def bound(case, side, t, err):
    _, b, s, h, hk, *_ = case
    items = [b * s * math.ceil(n / 4) for n in (h, hk)]
    blocks = [math.ceil(i / 4) for i in items]
    if sum(blocks) > 2 * SMS - 1:
        blocks = [max(1, i * (2 * SMS - 1) // sum(blocks)) for i in blocks]
    adds = math.ceil(items[side] / (4 * blocks[side])) + 2 + 4 + MOST_BLOCKS // 32 + 5
    return err.sum((0, 1, 2)) + adds * U * t.sum((0, 1, 2))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_what_is_lost_shows(case):
    """The bound is passed if any one item is missing or counted twice.  The mistake is made in the definition's sums."""
    x, dy, cos, sin, pos = inputs(case)
    for side in range(2):
        t, err = terms(case, x[side], dy[side], cos, sin, pos)
        w = bound(case, side, t, err)
        for h0 in range(0, t.shape[2], 4):
            lost = t[:, :, h0:h0 + 4].sum(2)
            assert np.all(np.any(lost > 2 * w, -1)), (side, h0)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_positive_terms(case):
    from tests.test_gpu_qk_norm import Problem
    dtype, b, s, h, hk, d, rot, inter = case
    p = Problem(dtype, b, s, h, hk, d, rot, inter, weights="32")
    x, dy, cos, sin, pos = inputs(case)
    p.x, p.dy = [p.place(t) for t in x], [p.place(t) for t in dy]
    if rot:
        p.cos.copy_(cos), p.sin.copy_(sin), p.pos.copy_(pos)
    _, dw, _ = p.bwd()
    for side in range(2):
        t, err = terms(case, x[side], dy[side], cos, sin, pos)
        off = np.abs(dw[side].double().cpu().numpy() - t.sum((0, 1, 2)))
        w = bound(case, side, t, err)
        assert np.all(off <= w), (side, float((off / w).max()))
