"""Head norms with the position rotation, the quantized key / value cache and
attention over it (oracle side).

TEST INFRASTRUCTURE ONLY - see the package docstring.

Norms, rotations, scores and sums are float64 on the exact input values.  The
cache's quantizers take their decisions in float32, one IEEE operation at a
time, as the other quantizers here do; the values that codes stand for are
float64 products.
"""

import numpy as np

from .formats import e4m3_decode, e4m3_encode, pack_u4, unpack_u4

F32 = np.float32
KV_SCALE_FLOOR = F32(2.0 ** -64)


def norm_rope(x, gamma, positions, inv_freq, eps, interleaved):
    """x [T][H][D] -> float64 [T][H][D]: RMSNorm per head (gamma None: none),
    then the rotation of the first 2 len(inv_freq) channels by the angle
    positions[t] * inv_freq[i]."""
    y = np.asarray(x, dtype=np.float64)
    if gamma is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)
    h = len(inv_freq)
    if h == 0:
        return y.copy()
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    out = y.copy()
    if interleaved:
        a, b = y[..., 0:2 * h:2], y[..., 1:2 * h:2]
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :h], y[..., h:2 * h]
        out[..., :h], out[..., h:2 * h] = a * c - b * s, b * c + a * s
    return out


def kv_quantize(x, fmt):
    """Rows x (float32 [..][D]) -> (codes, scales) as the cache holds them:
    int8 / uint8 codes and float32 scales, or packed uint8 codes and
    (fp16 scale, fp16 zero-point) pairs for "u4".  Rows with a NaN or an
    infinity: NaN scale, zero codes (and zero-point)."""
    x = np.asarray(x, dtype=np.float32)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], F32(0), x)
    if fmt == "u4":
        lo = np.minimum(x.min(axis=-1), F32(0))
        hi = np.maximum(x.max(axis=-1), F32(0))
        with np.errstate(over="ignore"):
            s = np.minimum(np.maximum(hi - lo, F32(1e-5)) / F32(15), F32(65504)).astype(np.float16)
        s32 = s.astype(np.float32)
        z = np.clip(np.rint(-lo / s32), 0, 15).astype(np.float32)
        n = np.clip(np.rint(x / s32[..., None]) + z[..., None], 0, 15).astype(np.uint8)
        n[bad] = 0
        pair = np.stack([s, z.astype(np.float16)], axis=-1)
        pair[bad] = [np.nan, 0]
        return pack_u4(n), pair
    a = np.abs(x).max(axis=-1)
    s = np.maximum(a / F32(127 if fmt == "int8" else 448), KV_SCALE_FLOOR)
    s = np.where(a == 0, F32(1), s).astype(np.float32)
    n = x / s[..., None]
    codes = np.rint(n).astype(np.int8) if fmt == "int8" else e4m3_encode(n)
    codes[bad] = 0
    s[bad] = np.nan
    return codes, s


def kv_values(codes, scales, fmt):
    """The float64 values that codes and scales stand for."""
    if fmt == "u4":
        n = unpack_u4(codes, 2 * codes.shape[-1]).astype(np.float64)
        sc = np.asarray(scales, dtype=np.float64)
        return (n - sc[..., 1:]) * sc[..., :1]
    n = codes.astype(np.float64) if fmt == "int8" else e4m3_decode(codes)
    return n * np.asarray(scales, dtype=np.float64)[..., None]


def tree_attention(q, k, v, seen, scale):
    """One sequence.  q [n][Hq][D], k, v [L][Hk][D] float64, seen bool [n][L].
    Returns (out, lse, weight, spread) with weight = sum p |v| (what rounding
    the probabilities can move) and spread = max over the seen tokens of
    scale sum |q k| (what rounding the scores can move)."""
    q = np.asarray(q, dtype=np.float64)
    n, hq, d = q.shape
    hk = k.shape[1]
    g = hq // hk
    out, weight = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, spread = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if at.size == 0:
            continue
        for h in range(hq):
            kk, vv = k[at, h // g], v[at, h // g]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            lse[i, h] = m + np.log(e.sum())
            out[i, h] = p @ vv
            weight[i, h] = p @ np.abs(vv)
            spread[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, weight, spread
