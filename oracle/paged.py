"""The paged cache and its attention by their definitions, in numpy: e4m3 numbers from the format (four exponent bits
of bias 7, three fraction bits, no infinities, 0x7f NaN), rows and places one by one, attention in 64 bits."""
import numpy as np

TOP, FLOOR = np.float32(448), np.float32(2.0 ** -110)


def _table():
    t = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = (8 + f) / 8 * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        if c & 127 == 127:
            x = np.nan
        t[c] = -x if c & 128 else x
    return t


E4M3 = _table()  # the number of every code


def to_code(x):
    """Codes of the e4m3 numbers nearest to x (ties to the even code; beyond 448: 448; NaN: a NaN code)."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    a = np.minimum(np.abs(x), 448.0)
    lo = np.searchsorted(mid, a, side="left")   # a tie stays below ..
    hi = np.searchsorted(mid, a, side="right")  # .. or goes above
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127 | (code & 128), code).astype(np.uint8)


def quantise(x):
    """(codes, fp32 scales) of rows x [..., d] of 16-bit values: the fp32 quotients and products the format is defined by."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.where(np.isfinite(x), np.abs(x), np.float32(0)).max(-1)
        a = np.maximum(a, FLOOR)
        up = (TOP / a).astype(np.float32)
        return to_code(x * up[..., None]), (a / TOP).astype(np.float32)


def values(codes, scales):
    """fp32 values of codes [..., d] with scales [...]."""
    with np.errstate(invalid="ignore", over="ignore"):
        return E4M3[codes].astype(np.float32) * np.asarray(scales, np.float32)[..., None]


def attention(q, k, v, scale, causal):
    """q [m, h, d] the last tokens of a sequence, k, v [n, h_kv, d] -> O [m, h, d], LSE [m, h], and for error bounds the
    weights P [m, h, n] and sum |q k| scale [m, h, n]."""
    m, h, d = q.shape
    n, hk = k.shape[:2]
    kk, vv = (np.repeat(t, h // hk, 1) for t in (k, v))
    s = np.einsum("mhd,nhd->mhn", q, kk) * scale
    mag = np.einsum("mhd,nhd->mhn", np.abs(q), np.abs(kk)) * abs(scale)
    seen = np.arange(n)[None, :] <= (np.arange(m) + n - m)[:, None] if causal else np.ones((m, n), bool)
    s = np.where(seen[:, None, :], s, -np.inf)
    top = s.max(-1, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0)[..., None])
    l = p.sum(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(l > 0, top + np.log(l), np.inf)
        p = np.where(l[..., None] > 0, p / l[..., None], 0)
    return np.einsum("mhn,nhd->mhd", p, vv), lse, p, np.where(seen[:, None, :], mag, 0), np.where(seen[:, None, :], s, 0)
