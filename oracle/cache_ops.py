"""64-bit forms of the operators around the attention path, in numpy: rotary positions, masked attention,
accumulated cache weights, eviction.  Test infrastructure, written from the formulas."""
import numpy as np


def voxel_positions(grid, voxel=None, offset=(0, 0, 0)):
    """int64 [N, 3] positions of a grid's tokens in raster order, or voxel by voxel."""
    T, H, W = grid
    out = []
    vt, vh, vw = voxel if voxel is not None else (1, 1, W)
    if voxel is None:
        out = [(t, h, w) for t in range(T) for h in range(H) for w in range(W)]
    else:
        for t0 in range(0, T, vt):
            for h0 in range(0, H, vh):
                for w0 in range(0, W, vw):
                    out += [(t, h, w) for t in range(t0, min(t0 + vt, T)) for h in range(h0, min(h0 + vh, H))
                            for w in range(w0, min(w0 + vw, W))]
    return np.asarray(out, dtype=np.int64) + np.asarray(offset, dtype=np.int64)


def rope(x, pos, axes, theta=10000.0, inv_freq=None, half=False, inverse=False):
    """x [B, H, N, d] float64, pos [N, A] or [B, N, A] whole numbers."""
    y = np.array(x, dtype=np.float64)
    pos = np.asarray(pos, dtype=np.float64)
    pos = pos[None] if pos.ndim == 2 else pos
    r, pair = sum(axes), 0
    for a, n in enumerate(axes):
        for i in range(n // 2):
            f = inv_freq[pair] if inv_freq is not None else theta ** (-2.0 * i / n)
            t = pos[:, None, :, a] * f * (-1.0 if inverse else 1.0)
            u, v = (pair, pair + r // 2) if half else (2 * pair, 2 * pair + 1)
            xu, xv = y[..., u].copy(), y[..., v].copy()
            y[..., u] = xu * np.cos(t) - xv * np.sin(t)
            y[..., v] = xu * np.sin(t) + xv * np.cos(t)
            pair += 1
    return y


def visible(Nq, Nk, causal=0, docs_q=None, docs_k=None, prefix=None, length=None):
    """(bool [Nq, Nk], float64 [Nq, Nk] distances) of one batch entry."""
    see = np.zeros((Nq, Nk), dtype=bool)
    dist = np.zeros((Nq, Nk))
    if docs_q is None:
        docs_q, docs_k = [0, Nq], [0, Nk if length is None else int(length)]
    for e in range(len(docs_q) - 1):
        k0, k1 = int(docs_k[e]), int(docs_k[e + 1])
        for i in range(int(docs_q[e]), min(int(docs_q[e + 1]), Nq)):
            p = (i - docs_q[e]) + (k1 - k0) - (docs_q[e + 1] - docs_q[e])
            c = np.arange(k1 - k0)
            ok = np.ones(k1 - k0, dtype=bool)
            if causal:
                ok = c // causal <= p // causal
                if prefix is not None:
                    ok |= c < prefix[e]
            see[i, k0:k1] = ok
            dist[i, k0:k1] = np.abs(p - c)
    return see, dist


def scores(q, k, scale, cap=0.0, slope=0.0, dist=None):
    s = scale * (q @ k.T)
    if cap:
        s = cap * np.tanh(s / cap)
    return s - slope * dist if slope else s


def attention(q, k, v, scale, see, **mods):
    """One head: (o, lse, sum of p |v|, largest scale * sum |q k| over what is seen)."""
    s = np.where(see, scores(q, np.where(see.any(0)[:, None], k, 0.0), scale, **mods), -np.inf)
    m = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    m = np.where(np.isinf(m), 0.0, m)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    some = l[:, 0] > 0
    p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    v = np.where(see.any(0)[:, None], v, 0.0)
    o = p @ v
    with np.errstate(divide="ignore"):
        lse = np.where(some, np.log(l[:, 0]) + m[:, 0], -np.inf)
    return o, lse, p @ np.abs(v)


def cache_weights(q, k, lse, scale, see, **mods):
    """One query head's sum over rows of e^(s - lse): [Nk]."""
    k = np.where(see.any(0)[:, None], k, 0.0)
    live = np.isfinite(lse)
    s = scores(np.where(live[:, None], q, 0.0), k, scale, **mods)
    p = np.exp(np.where(see & live[:, None], s - np.where(live, lse, 0.0)[:, None], -np.inf))
    return p.sum(0)


def evict(w, n, budget, sink, recent):
    """Kept entries of one head's n, ascending."""
    w = np.asarray(w, dtype=np.float64)[:n]
    if n <= budget:
        return np.arange(n)
    mid = np.arange(sink, n - recent)
    key = np.where(np.isnan(w[mid]), -np.inf, w[mid]) + 0.0
    nan = np.isnan(w[mid])
    order = np.lexsort((mid, nan, -key))  # larger first, numbers before NaN, then the lower index
    want = budget - sink - recent
    return np.sort(np.concatenate([np.arange(sink), mid[order[:want]], np.arange(n - recent, n)]))
