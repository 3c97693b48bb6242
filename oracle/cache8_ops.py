"""64-bit forms of the normalised rotation, its gradient, and the 8-bit key-value cache, in numpy.  Test infrastructure,
written from the formulas."""
import numpy as np

from oracle import cache_ops as O


def normalised(x, layer, eps):
    """(n, 1 / deviation) over the last axis."""
    mu = x.mean(-1, keepdims=True) if layer else 0.0
    r = 1.0 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    return (x - mu) * r, r


def norm_rope(x, pos, axes, layer=False, eps=1e-6, w=None, b=None, **rope):
    y = normalised(x, layer, eps)[0]
    y = y * (1.0 if w is None else w) + (0.0 if b is None else b)
    return O.rope(y, pos, axes, **rope)


def norm_rope_grad(dy, x, pos, axes, layer=False, eps=1e-6, w=None, **rope):
    """(dx, dw, db)."""
    n, r = normalised(x, layer, eps)
    g = O.rope(dy, pos, axes, inverse=True, **rope)
    h = g * (1.0 if w is None else w)
    dx = h - n * (h * n).mean(-1, keepdims=True)
    if layer:
        dx = dx - h.mean(-1, keepdims=True)
    return dx * r, (g * n).sum((0, 1, 2)), g.sum((0, 1, 2))


# every code's value: sign, four exponent bits (bias 7, 0: steps of 2^-9), three of the mantissa; 0x7F and 0xFF are NaN
_e, _m = np.arange(128) >> 3, np.arange(128) & 7
_VALUES = np.where(_e > 0, (1 + _m / 8.0) * 2.0 ** (_e - 7.0), _m * 2.0 ** -9)
_VALUES[127] = np.nan
VALUES = np.concatenate([_VALUES, -_VALUES])


def decode(codes):
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def encode(x):
    """The nearest code of each value (|x| <= 464; ties to the even code, what is not finite to NaN)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    grid = _VALUES[:127]
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isfinite(x), code, 127)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(top):
    """The least power of two, 2^-126 at least, that brings top to 448 or below; 0 for 0."""
    if top == 0:
        return 0.0
    e = -126
    while top / 2.0 ** e > 448:
        e += 1
    return 2.0 ** e


def held(s):
    return float(s) if np.isfinite(s) and s > 0 else 0.0


def values(codes, scales, block):
    """A head's [N, d] codes and [blocks] scales as values."""
    per = np.array([held(s) for s in scales])[np.arange(codes.shape[0]) // block][:, None]
    return np.where(per > 0, decode(codes) * per, 0.0)


def append(codes, scales, new, start, count, block):
    """One head's cache after the call: (codes, scales), and which of them the call defines (bool like both)."""
    codes, scales = codes.copy(), np.array(scales, dtype=np.float64)
    N = codes.shape[0]
    i0, i1 = max(start, 0), min(start + count, N)
    for j in range(i0 // block, -(-i1 // block) if i1 > i0 else 0):
        t0, t1 = j * block, min(N, (j + 1) * block)
        w0, w1 = max(t0, i0), min(t1, i1)
        x = new[w0 - start:w1 - start]
        fin = np.abs(np.where(np.isfinite(x), x, 2.0 ** -149))
        old = 0.0 if (w0, w1) == (t0, t1) else held(scales[j])
        s = max(old, scale_for(fin.max(initial=0.0)))
        if s != old:
            for t in list(range(t0, w0)) + list(range(w1, t1)):
                codes[t] = encode(decode(codes[t]) * old / s) if old else 0
        codes[w0:w1] = encode(x / s) if s else encode(x)
        scales[j] = s
    return codes, scales


def attention(q, k, v, scale, hi):
    """One head's rows q [n, d], row i over keys 0 .. hi[i] - 1: (o, lse, sum of p |v|, largest scale sum |q k|)."""
    see = np.arange(k.shape[0])[None] < np.asarray(hi)[:, None]
    return O.attention(q, k, v, scale, see) + (abs(scale) * float((np.abs(q) @ np.where(see.any(0)[:, None], np.abs(k), 0.0).T).max(initial=0.0)),)


def row_ends(Nq, n, causal):
    """How many keys each row sees of n: the rows are the last positions."""
    p = np.arange(Nq) + n - Nq
    return np.clip((p // causal + 1) * causal, 0, n) if causal else np.full(Nq, n)
