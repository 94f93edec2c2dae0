"""Plain implementations in 64 bits and more of the operators that check
drafted tokens (rotation with the cache write, attention of a tree, the draw of
a token), for the tests.

Stored codes are decoded by the C oracle.  Nothing here shares code with the
kernels or the binding.
"""
import numpy as np

import serving_model as model


def turns(positions, freqs, axes=None):
    """(cos, sin) [tokens, n] in extended precision of position * freq."""
    p = np.asarray(positions).astype(np.longdouble)
    f = np.asarray(freqs, dtype=np.float32).astype(np.longdouble)
    p = p[:, None] if axes is None else p[np.minimum(np.asarray(axes).astype(np.int64), len(p) - 1)].T
    angle = p * f
    return np.cos(angle), np.sin(angle)


def rotate(x, cos, sin, interleaved):
    """(y, span) of float64 x [tokens, heads, D]: the rotated rows, and |a| + |b| of each element's pair (0: not turned)."""
    n = cos.shape[1]
    x = np.asarray(x, dtype=np.float64)
    y, span = x.copy(), np.zeros_like(x)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., first].astype(np.longdouble), x[..., second].astype(np.longdouble)
    c, s = cos[:, None], sin[:, None]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    span[..., first] = span[..., second] = np.abs(a) + np.abs(b)
    return y, span


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1_round(v):
    """E2M1 value of float64 v, ties to the even code.  Monotone in v."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    quantum = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.sign(v) * np.rint(a / quantum) * quantum


def e2m1_decode(q):
    """float64 values of packed codes, element 2 j in the low nibble."""
    q = np.asarray(q)
    c = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def check_codes(q, s, y, span, fmt, what=""):
    """(q, s) [..., D] are codes of some y' with |y' - y| <= span: the scale is that
    of a largest magnitude in the interval, and every element lies between the
    codes of the interval's ends (rounding and saturation are monotone)."""
    top = 8 if fmt == "mxfp8" else 2
    b, w = (a.reshape(*a.shape[:-1], -1, 32) for a in (y, span))

    def exponent(a):
        return np.where(a > 0, np.clip(np.frexp(a)[1] - 1 - top, -127, 127), -127)

    e = np.asarray(s).astype(np.int64) - 127
    lo = exponent(np.maximum(np.abs(b) - w, 0).max(axis=-1))
    hi = exponent((np.abs(b) + w).max(axis=-1))
    bad = (e < lo) | (e > hi)
    assert not bad.any(), f"{what}: {int(bad.sum())} scales off, first at {np.argwhere(bad)[0]}"
    scale = np.exp2(-e.astype(np.float64))[..., None]
    got = (model.e4m3_decode(q) if fmt == "mxfp8" else e2m1_decode(q)).reshape(b.shape)
    rnd = model.e4m3_round if fmt == "mxfp8" else e2m1_round
    bad = ~((got >= rnd((b - w) * scale)) & (got <= rnd((b + w) * scale)))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {np.argwhere(bad)[0]}"
