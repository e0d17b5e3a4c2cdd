"""fp64 definitions of the position operators (numpy): the norm and rotation of query / key heads with its
gradient, and attention with a learned relative position bias by buckets.  Shares nothing with the CUDA
code; inputs are the exact 16-bit values widened to fp64.

Tensors are token-major [b, s, h, d].
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------- norm and rotation

def _turn(z, cos, sin, rot, interleaved):
    """z [b, s, h, d] turned by the angles whose cos / sin [b, s, rot / 2] are given."""
    out = z.copy()
    if rot == 0:
        return out
    c, s = cos[:, :, None, :], sin[:, :, None, :]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = z[..., ia], z[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def norm_rope(x, w, eps, cos, sin, rot, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, cos, sin, rot, interleaved)


def norm_rope_bwd(x, dy, w, eps, cos, sin, rot, interleaved):
    """(dx, dw)"""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dz = _turn(dy, cos, None if sin is None else -sin, rot, interleaved)
    g = dz * w
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), (dz * xh).sum((0, 1, 2))


# --------------------------------------------------------------------------- relative position bias

def bucket(delta, num_buckets, max_distance, bidirectional):
    """Bucket of a key `delta` positions after its query, by integer comparison: past the exact buckets,
    distance x has reached step m when (x / e)^(n - e) >= (max_distance / e)^m."""
    n = num_buckets // 2 if bidirectional else num_buckets
    base = n if bidirectional and delta > 0 else 0
    x = abs(delta) if bidirectional else max(-delta, 0)
    e = n // 2
    if x < e:
        return base + x
    x = min(x, max_distance)
    m = 0
    while e + m < n - 1 and x ** (n - e) * e ** (m + 1) >= max_distance ** (m + 1) * e ** (n - e):
        m += 1
    return base + e + m


def bucket_matrix(s_q, s_kv, shift, num_buckets, max_distance, bidirectional):
    d = np.arange(s_kv)[None, :] - np.arange(s_q)[:, None] - shift
    lo = int(d.min()) if d.size else 0
    hi = int(d.max()) if d.size else 0
    tab = np.array([bucket(x, num_buckets, max_distance, bidirectional) for x in range(lo, hi + 1)], np.int64)
    return tab[d - lo]


MASKED = -1e30  # a table entry at or below this masks its bucket out


def _scores(q, k, table_h, buckets, scale, mask, shift):
    """Scores [s_q, s_kv] of one head, -inf where the key is not visible."""
    s = scale * (q @ k.T) + table_h[buckets]
    hide = table_h[buckets] <= MASKED
    i, j = np.arange(s.shape[0])[:, None], np.arange(s.shape[1])[None, :]
    if mask:  # 1: top-left, 2: bottom-right
        hide = hide | (j > i + shift)
    return np.where(hide, -np.inf, s)


def _shift(mask, s_q, s_kv):
    return s_kv - s_q if mask == 2 else 0


def relbias_fwd(q, k, v, table, scale, mask, max_distance, bidirectional):
    """One sequence: q [s_q, h, d], k, v [s_kv, h_kv, d], table [buckets, h] -> O [s_q, h, d], LSE [s_q, h]."""
    sq, h, d = q.shape
    sk, hk = k.shape[:2]
    sh = _shift(mask, sq, sk)
    bk = bucket_matrix(sq, sk, sh, table.shape[0], max_distance, bidirectional)
    o, lse = np.zeros((sq, h, d)), np.full((sq, h), np.inf)
    for x in range(h):
        g = x // (h // hk)
        s = _scores(q[:, x], k[:, g], table[:, x], bk, scale, mask, sh)
        m = s.max(-1, initial=-np.inf)
        live = m > -np.inf
        p = np.exp(s[live] - m[live, None])
        l = p.sum(-1)
        o[live, x] = (p @ v[:, g]) / l[:, None]
        lse[live, x] = m[live] + np.log(l)
    return o, lse


def relbias_bwd(q, k, v, o, do, lse, table, scale, mask, max_distance, bidirectional):
    """One sequence, from the supplied O and LSE [s_q, h]: dQ, dK, dV, dtable."""
    sq, h, d = q.shape
    sk, hk = k.shape[:2]
    sh = _shift(mask, sq, sk)
    bk = bucket_matrix(sq, sk, sh, table.shape[0], max_distance, bidirectional)
    dq, dk, dv, dt = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(table)
    for x in range(h):
        g = x // (h // hk)
        s = _scores(q[:, x], k[:, g], table[:, x], bk, scale, mask, sh)
        p = np.exp(np.where(np.isneginf(s), -np.inf, s - np.where(np.isinf(lse[:, x]), 0.0, lse[:, x])[:, None]))
        p[np.isinf(lse[:, x])] = 0.0
        ds = p * (do[:, x] @ v[:, g].T - (do[:, x] * o[:, x]).sum(-1, keepdims=True))
        dv[:, g] += p.T @ do[:, x]
        dk[:, g] += scale * ds.T @ q[:, x]
        dq[:, x] = scale * ds @ k[:, g]
        np.add.at(dt[:, x], bk, ds)
    return dq, dk, dv, dt
