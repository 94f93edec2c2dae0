"""Plain float64 implementations of the serving operators (norm with MXFP8
output, paged MX cache, attention of one new token), for the tests.

Stored codes are decoded by the C oracle.  Nothing here shares code with the
kernels or the binding.
"""
import numpy as np

import oracle


def bf16_round(x):
    """float64 -> nearest bf16 value (ties to even), as float64; normal range."""
    u = np.asarray(x, dtype=np.float64).view(np.uint64)
    r = (u + np.uint64((1 << 44) - 1) + ((u >> np.uint64(45)) & np.uint64(1))) & ~np.uint64((1 << 45) - 1)
    return r.view(np.float64)


def e4m3_round(v):
    """E4M3 value of float64 v: quantum 2^(max(floor log2 |v|, -6) - 3), half
    to even, saturating at 448.  Monotone in v."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -30))
    quantum = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(v / quantum) * quantum, -448.0, 448.0)


def e4m3_decode(q):
    table = np.array([oracle.e4m3_decode(c) for c in range(256)])
    return table[np.asarray(q)]


def norm_rows(x, residual, weight, eps, bf16):
    """(r, y) in float64: r rounded to the stored type, y the normalised rows."""
    r = x if residual is None else x + residual
    if residual is not None:
        r = bf16_round(r) if bf16 else r.astype(np.float32).astype(np.float64)
    return r, r / np.sqrt((r * r).mean(axis=-1, keepdims=True) + eps) * weight


def check_mx8(q, s, y, delta, what=""):
    """(q, s) are MXFP8 codes of some y' with |y' - y| <= delta |y|: the scale
    is that of an amax in the interval, and every element lies between the
    codes of the interval's ends (rounding and saturation are monotone)."""
    rows, k = y.shape
    b = y.reshape(rows, k // 32, 32)
    amax = np.abs(b).max(axis=-1)

    def exponent(a):
        return np.where(a > 0, np.clip(np.frexp(a)[1] - 1 - 8, -127, 127), -127)

    e = s.astype(np.int64) - 127
    lo, hi = exponent(amax * (1 - delta)), exponent(amax * (1 + delta))
    bad = (e < lo) | (e > hi)
    assert not bad.any(), f"{what}: {int(bad.sum())} scales off, first at {np.argwhere(bad)[0]}"
    scale = np.exp2(-e.astype(np.float64))[..., None]
    got = e4m3_decode(q).reshape(b.shape)
    span = np.abs(b) * delta
    low, high = e4m3_round((b - span) * scale), e4m3_round((b + span) * scale)
    bad = ~((got >= low) & (got <= high))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {np.argwhere(bad)[0]}"


def quantize_rows(x, fmt):
    return oracle.mx8_quantize(x) if fmt == "mxfp8" else oracle.mx_quantize(x)


def dequantize_rows(q, s, fmt):
    return oracle.mx8_dequantize(q, s) if fmt == "mxfp8" else oracle.mx_dequantize(q, s)


def token_rows(cache, page, pos, fmt):
    """float64 keys and values [heads, D] of one slot of a host cache."""
    kq, ks, vq, vs = cache
    return (dequantize_rows(np.ascontiguousarray(kq[page, :, pos]), np.ascontiguousarray(ks[page, :, pos]), fmt),
            dequantize_rows(np.ascontiguousarray(vq[page, :, pos]), np.ascontiguousarray(vs[page, :, :, pos]), fmt))


def attention(q, cache, table, lens, fmt, scale, window=0, sinks=None):
    """(out, weight_sum) in float64, [batch, q_heads, D]: out by the
    definition, and sum_t p_t |V_t| / denominator, the size its error bound
    scales with; also the largest error factor of a score, per (batch, head):
    sum_d |q_d K_d| * |scale|."""
    q = np.asarray(q, dtype=np.float64)
    batch, heads, d = q.shape
    pages, hkv, page = cache[0].shape[:3]
    out, size = np.zeros_like(q), np.zeros_like(q)
    mag = np.zeros((batch, heads))
    for b in range(batch):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        at = [t for t in range(max(0, n - window) if window else 0, n) if 0 <= table[b, t // page] < pages]
        if not at:
            continue
        rows = [token_rows(cache, table[b, t // page], t % page, fmt) for t in at]
        k = np.stack([r[0] for r in rows])  # [t, hkv, d]
        v = np.stack([r[1] for r in rows])
        for h in range(heads):
            kh, vh = k[:, h // (heads // hkv)], v[:, h // (heads // hkv)]
            s = kh @ q[b, h] * scale
            mag[b, h] = (np.abs(kh) @ np.abs(q[b, h])).max() * abs(scale)
            top = max(s.max(), sinks[h]) if sinks is not None else s.max()
            p = np.exp(s - top)
            total = p.sum() + (np.exp(sinks[h] - top) if sinks is not None else 0.0)
            out[b, h] = p @ vh / total
            size[b, h] = p @ np.abs(vh) / total
    return out, size, mag
