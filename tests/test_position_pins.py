"""Pins of the fp64 position-operator definitions (oracle/position.py): central differences, orthogonality of
the rotation, bucket borders worked by hand, and the equality with plain attention where the bias is
constant."""
import numpy as np
import pytest

import oracle
from oracle import position as P


def _angles(rng, b, s, rot):
    if rot == 0:
        return None, None
    a = rng.uniform(-3, 3, (b, s, rot // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (16, True), (32, False), (32, True)])
def test_norm_rope_gradient_against_differences(rot, interleaved):
    rng = np.random.default_rng(rot + interleaved)
    x, dy, w = rng.normal(size=(2, 3, 2, 32)), rng.normal(size=(2, 3, 2, 32)), rng.normal(size=32)
    cos, sin = _angles(rng, 2, 3, rot)
    f = lambda x, w: (P.norm_rope(x, w, 1e-3, cos, sin, rot, interleaved) * dy).sum()
    dx, dw = P.norm_rope_bwd(x, dy, w, 1e-3, cos, sin, rot, interleaved)
    e = 1e-5
    for idx in [(0, 0, 0, 0), (1, 2, 1, 31), (0, 1, 1, 8), (1, 0, 0, 17)]:
        p = x.copy(); p[idx] += e
        m = x.copy(); m[idx] -= e
        assert abs((f(p, w) - f(m, w)) / (2 * e) - dx[idx]) < 1e-8
    for c in (0, 7, 8, 31):
        p = w.copy(); p[c] += e
        m = w.copy(); m[c] -= e
        assert abs((f(x, p) - f(x, m)) / (2 * e) - dw[c]) < 1e-8


def test_rotation_by_hand():
    """One pair turned by 90 degrees: (a, b) -> (-b, a); the two pairings; what is not rotated stays."""
    x = np.arange(1.0, 33.0).reshape(1, 1, 1, 32)
    r = 1 / np.sqrt((x * x).mean())
    c, s = np.zeros((1, 1, 8)), np.ones((1, 1, 8))
    y = P.norm_rope(x, np.ones(32), 0.0, c, s, 16, False)[0, 0, 0] / r
    np.testing.assert_allclose(y[:16], np.concatenate([-np.arange(9.0, 17.0), np.arange(1.0, 9.0)]), rtol=1e-14)
    np.testing.assert_allclose(y[16:], np.arange(17.0, 33.0), rtol=1e-14)
    y = P.norm_rope(x, np.ones(32), 0.0, c, s, 16, True)[0, 0, 0] / r
    np.testing.assert_allclose(y[:4], [-2, 1, -4, 3], rtol=1e-14)


def test_buckets_by_hand():
    """32 buckets to distance 128, both directions: 8 exact distances a side, then steps at 8 * 2^(m / 2)."""
    got = [P.bucket(-x, 32, 128, True) for x in (0, 7, 8, 11, 12, 15, 16, 22, 23, 31, 32, 90, 91, 127, 128, 5000)]
    assert got == [0, 7, 8, 8, 9, 9, 10, 10, 11, 11, 12, 14, 15, 15, 15, 15]
    assert P.bucket(1, 32, 128, True) == 17 and P.bucket(5000, 32, 128, True) == 31
    # one direction: 16 exact, then steps at 16 * 8^(m / 16); keys after the query share bucket 0
    assert [P.bucket(-x, 32, 128, False) for x in (0, 15, 16, 18, 19, 112, 113, 128)] == [0, 15, 16, 16, 17, 30, 31, 31]
    assert P.bucket(3, 32, 128, False) == 0


@pytest.mark.parametrize("mask", [0, 1, 2])
@pytest.mark.parametrize("sq,sk,h,hk", [(5, 5, 2, 2), (4, 9, 4, 2), (9, 4, 2, 1), (1, 7, 2, 2)])
def test_relbias_gradients_against_differences(mask, sq, sk, h, hk):
    rng = np.random.default_rng(17 * mask + sq)
    d, nb = 4, 8
    q, k, v = rng.normal(size=(sq, h, d)), rng.normal(size=(sk, hk, d)), rng.normal(size=(sk, hk, d))
    do, t = rng.normal(size=(sq, h, d)), rng.normal(size=(nb, h))
    kw = dict(scale=0.7, mask=mask, max_distance=6, bidirectional=True)
    o, lse = P.relbias_fwd(q, k, v, t, **kw)
    grads = P.relbias_bwd(q, k, v, o, do, lse, t, **kw)
    f = lambda a: (P.relbias_fwd(*a, **kw)[0] * do).sum()
    e = 1e-5
    for n, g in enumerate(grads):
        for idx in np.ndindex(g.shape):
            p = [x.copy() for x in (q, k, v, t)]
            m = [x.copy() for x in (q, k, v, t)]
            p[n][idx] += e
            m[n][idx] -= e
            assert abs((f(p) - f(m)) / (2 * e) - g[idx]) < 1e-7


def test_constant_bias_is_plain_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(6, 2, 8)), rng.normal(size=(6, 2, 8)), rng.normal(size=(6, 2, 8))
    t = np.full((16, 2), 0.75)
    o, lse = P.relbias_fwd(q, k, v, t, 0.5, 2, 20, False)
    ro, rl = oracle.dense_fwd(q, k, v, np.array([6]), np.array([6]), 0.5, oracle.CAUSAL_BOTTOM_RIGHT)
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(lse, rl + 0.75, atol=1e-13)


def test_masked_bucket_hides_its_keys():
    """A row whose only bucket is masked sees no key; others lose that bucket's keys alone."""
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(3, 1, 4)), rng.normal(size=(3, 1, 4)), rng.normal(size=(3, 1, 4))
    t = rng.normal(size=(8, 1))
    t[0] = -np.inf  # distance 0, one direction
    o, lse = P.relbias_fwd(q, k, v, t, 1.0, 2, 20, False)
    assert np.all(o[0] == 0) and np.isposinf(lse[0, 0])
    np.testing.assert_allclose(o[1, 0], v[0, 0], atol=1e-14)
    dq, dk, dv, dt = P.relbias_bwd(q, k, v, o, rng.normal(size=(3, 1, 4)), lse, t, 1.0, 2, 20, False)
    assert np.all(dq[0] == 0) and np.all(dk[2] == 0) and dt[0, 0] == 0 and np.all(np.isfinite(dt))
