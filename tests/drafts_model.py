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


# ------------------------------------------------------------------ attention of a tree

def bits_of(mask):
    """Truth values [batch, drafts, drafts] of masks [batch, drafts, words] of 64 bits."""
    m = np.ascontiguousarray(mask).view(np.uint64)
    drafts = m.shape[1]
    at = np.arange(drafts)
    return (m[:, :, at // 64] >> (at % 64).astype(np.uint64)) & np.uint64(1) != 0


def mask_of(bits):
    """The reverse: int64 words."""
    bits = np.asarray(bits, dtype=bool)
    batch, drafts = bits.shape[:2]
    words = -(-drafts // 64)
    wide = np.zeros((batch, drafts, 64 * words), dtype=np.uint64)
    wide[:, :, :drafts] = bits
    return (wide.reshape(batch, drafts, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)


def visible(context, bits, table_row, pages, page, window=0, first=0):
    """What the tokens of one sequence see: truth values [drafts, n] over cache positions."""
    drafts = len(bits)
    most = len(table_row) * page
    n = min(max(int(context), 0), most)
    end = min(n + drafts, most)
    depth = np.array([bits[i, :i].sum() for i in range(drafts)])
    see = np.zeros((drafts, end), dtype=bool)
    place = np.concatenate((np.arange(n), n + depth))[:end]
    see[:, :n] = True
    see[:, n:] = bits[:, :end - n]
    if window:
        see &= ((n + depth)[:, None] - place[None] < window) | (place[None] < first)
    named = (table_row >= 0) & (table_row < pages)
    return see & named[np.arange(end) // page][None]


def tree_attention(q, cache, table, context, bits, fmt, scale, window=0, first=0, sinks=None):
    """(out, size, mag) in float64 as serving_model.attention, for q [batch, drafts, heads, D]."""
    q = np.asarray(q, dtype=np.float64)
    batch, drafts, heads, d = q.shape
    pages, hkv, page = cache[0].shape[:3]
    out, size, mag = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3])
    group = heads // hkv
    for b in range(batch):
        see = visible(context[b], bits[b], table[b], pages, page, window, first)
        at = np.flatnonzero(see.any(0))
        if not len(at):
            continue
        see = see[:, at]
        pg, pos = table[b, at // page], at % page
        kq, ks, vq, vs = cache
        vst = vs.transpose(0, 3, 1, 2)
        rows = []
        for c, s in ((kq[pg, :, pos], ks[pg, :, pos]), (vq[pg, :, pos], vst[pg, pos])):
            x = model.dequantize_rows(np.ascontiguousarray(c).reshape(-1, c.shape[-1]),
                                      np.ascontiguousarray(s).reshape(-1, s.shape[-1]), fmt)
            rows.append(np.asarray(x, dtype=np.float64).reshape(len(at), hkv, d))
        for h in range(heads):
            k, v = (r[:, h // group] for r in rows)
            s = np.where(see, (q[b, :, h] @ k.T) * scale, -np.inf)
            mag[b, :, h] = np.where(see, np.abs(q[b, :, h]) @ np.abs(k).T, 0).max(1) * abs(scale)
            some = see.any(1)
            top = np.where(some, s.max(1), 0.0)
            if sinks is not None:
                top = np.where(some, np.maximum(top, sinks[h]), 0.0)
            p = np.exp(s - top[:, None])
            total = p.sum(1) + (np.exp(sinks[h] - top) if sinks is not None else 0.0)
            total = np.where(some, total, 1.0)
            out[b, :, h] = p @ v / total[:, None]
            size[b, :, h] = p @ np.abs(v) / total[:, None]
    return out, size, mag


# ------------------------------------------------------------------ the draw of a token

def draw_check(x, u, temperature, top_k, top_p, min_p, token, share, what=""):
    """(token, share) is a right answer for one row of float64 logits.

    The weights are formed in extended precision.  The library's are whole
    multiples of 2^-43 of the largest (half of one off at most), from fp64 values
    within 2^-48: a sum over n of them is within n 2^-44 + 2^-48 of the sum, in
    units of the largest weight.  Where a threshold lies that close to a prefix's
    weight, either prefix is right, and either token where u's product lies that
    close to a running sum."""
    x = np.asarray(x, dtype=np.float64)
    n = len(x)
    if np.isnan(x).any() or x.max() == np.inf or x.max() == -np.inf:
        assert token == -1 and np.isnan(share), what
        return
    if not temperature > 0:
        assert token == int(np.argmax(x)) and share == 1, f"{what}: {token} for the largest {int(np.argmax(x))}"
        return
    with np.errstate(invalid="ignore"):
        z = (x - x.max()).astype(np.longdouble) / np.longdouble(np.float32(temperature))
    w = np.exp(np.where(np.isnan(z), -np.inf, z))
    order = np.lexsort((np.arange(n), -x))
    k = top_k if 0 < top_k < n else n
    sums = np.cumsum(w[order])
    off = n * 2.0 ** -44 + 2.0 ** -48 * float(sums[-1])
    lengths = {k}
    if np.float32(top_p) < 1:
        goal = np.longdouble(np.float32(top_p)) * sums[k - 1]
        lengths = {max(1, min(k, int(np.searchsorted(sums[:k], goal + d, side="left")) + 1)) for d in (-off, 0, off)}
    least = np.longdouble(min(np.float32(min_p), np.float32(1)))
    sizes = {max(1, int((w >= least + d).sum())) for d in (-2.0 ** -48, 0, 2.0 ** -48)}
    u = min(max(float(np.float32(u)), 0.0), 1.0)
    for length in lengths:
        for size in sizes:
            kept = np.zeros(n, dtype=bool)
            kept[order[:min(length, size)]] = True
            run = np.cumsum(np.where(kept, w, 0))
            total = run[-1]
            if 0 <= token < n and kept[token] and w[token] > 0:
                before = run[token] - w[token]
                if before - off <= u * total <= run[token] + off and (u < 1 or total - run[token] <= off):
                    # the share: fp64 weight, the sum off by `off`, one rounding
                    assert abs(share - w[token] / total) <= w[token] / total * (2.0 ** -23 + 2 * off / total), what
                    return
    raise AssertionError(f"{what}: token {token} (share {share}) is not the draw for u {u}, lengths {sorted(lengths)}")
