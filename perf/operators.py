"""The cache-and-position operators around the attention path, as cases that can be timed and compared.

Four operators of a video transformer that generates frame by frame over a rolling key-value window:

  rope     rotary positions of queries and keys along time, height and width, and the rotation's gradient
  masked   attention with frame-causal, document and prefix masks, scores capped by a tanh, a bias that falls
           with distance; many query rows, or one new token over a long cache
  weights  the attention weight that every cached key has received, accumulated over steps
  evict    the eviction of the least attended keys from the cache

`run` computes a case in plain tensor operations (own = False), or through the library's entry points (own = True).
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the 69K-token latent of a 720p clip, queries and keys of one layer in voxel order
        dict(name="rope_video69k", op="rope", B=1, H=24, Hk=24, d=128, axes="44,42,42", grid="18,48,80", voxel="2,8,8",
             offset=0, pairing="interleaved", dtype="bf16", layout="bhnd", inverse=False),
        # one chunk of 8 frames of 22x40 tokens entering a rolling window, straight from the projections (token-major)
        dict(name="rope_chunk", op="rope", B=1, H=12, Hk=12, d=128, axes="44,42,42", grid="8,22,40", voxel="",
             offset=24, pairing="interleaved", dtype="bf16", layout="bnhd", inverse=False),
        # the gradient at explicit positions (an image's two axes), fp32, an odd number of tokens: latency
        dict(name="rope_gradient_fp32", op="rope", B=2, H=3, Hk=0, d=64, axes="32,32", grid="1237", voxel="",
             offset=0, pairing="half", dtype="fp32", layout="bhnd", inverse=True),
        # a chunk's queries over the whole window; a frame sees itself and what came before
        dict(name="masked_frames", op="masked", B=1, H=12, Hk=12, d=128, Nq=7040, Nk=28160, causal=880, cap=0.0,
             bias=False, docs_q="", docs_k="", prefix="", layout="bhnd"),
        # clips of different lengths packed into one row, each after its text (a prefix all of it may see), capped scores
        dict(name="masked_packed_capped", op="masked", B=1, H=24, Hk=24, d=128, Nq=16384, Nk=16384, causal=1, cap=50.0,
             bias=False, docs_q="0,5000,5384,11001,11002,16384", docs_k="0,5000,5384,11001,11002,16384",
             prefix="226,0,511,1,226", layout="bnhd"),
        # shared key heads, a bias by distance, an odd length
        dict(name="masked_bias_shared", op="masked", B=2, H=16, Hk=4, d=64, Nq=4099, Nk=4099, causal=1, cap=0.0,
             bias=True, docs_q="", docs_k="", prefix="", layout="bhnd"),
        # one new token per sequence over caches of different fill, capped, shared key heads
        dict(name="masked_token", op="masked", B=4, H=24, Hk=6, d=128, Nq=1, Nk=28160, causal=1, cap=30.0, bias=False,
             docs_q="0,1;0,1;0,1;0,1", docs_k="0,28160;0,7041;0,20000;0,27999", prefix="", layout="bhnd"),
        # one new token over a single frame: latency
        dict(name="masked_token_frame", op="masked", B=1, H=12, Hk=12, d=128, Nq=1, Nk=880, causal=0, cap=0.0,
             bias=False, docs_q="", docs_k="", prefix="", layout="bhnd"),
        # the weight that a chunk's queries gave to every key of the window and of the chunk itself
        dict(name="weights_chunk", op="weights", B=1, H=12, Hk=12, d=128, Nq=7040, Nk=35200, causal=880, decay=0.9,
             lengths="", layout="bhnd"),
        # the same after one token per sequence
        dict(name="weights_token", op="weights", B=4, H=24, Hk=6, d=128, Nq=1, Nk=28160, causal=0, decay=1.0,
             lengths="28160,7041,20000,27999", layout="bhnd"),
        # a full window plus a chunk, cut back to the window; the first and the newest chunk stay
        dict(name="evict_window", op="evict", B=1, Hk=12, d=128, Nk=35200, budget=28160, sink=7040, recent=7040,
             lengths="", layout="bhnd"),
        # small caches of different fill, one of them under the budget: latency
        dict(name="evict_small", op="evict", B=3, Hk=5, d=64, Nk=2011, budget=733, sink=4, recent=64,
             lengths="2011,500,1500", layout="bnhd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _docs(rng, B, N, n):
    rows = []
    for _ in range(B):
        cuts = sorted(rng.randint(0, N) for _ in range(n - 1))
        rows.append([0] + cuts + [N])
    return rows


def _text(rows):
    return ";".join(",".join(str(x) for x in r) for r in rows)


def draw(rng):
    op = rng.choice(["rope", "masked", "masked", "weights", "evict"])
    d = rng.choice([64, 128])
    layout = rng.choice(["bhnd", "bnhd"])
    B = rng.choice([1, 1, 2, 3])
    if op == "rope":
        H = rng.choice([1, 3, 12, 24])
        pairing = rng.choice(["interleaved", "half"])
        three = rng.random() < 0.7
        if three:
            grid = [rng.randint(1, 12), rng.randint(1, 45), rng.randint(1, 80)]
            axes = {128: rng.choice(["44,42,42", "32,48,48"]), 64: "24,20,20"}[d]
            voxel = rng.choice(["", "2,8,8", "3,5,4"])
        else:
            grid, axes, voxel = [_log(rng, 1, 40000)], rng.choice(["%d" % d, "32,32", "16,24,24"]), ""
        Hk, dtype = rng.choice([0, 1, H]), rng.choice(["bf16", "bf16", "fp32"])
        most = 800_000_000 // (B * (H + Hk) * d * (4 if dtype == "fp32" else 2) * math.prod(grid[1:]))
        grid[0] = max(1, min(grid[0], most))
        return dict(op=op, B=B, H=H, Hk=Hk, d=d, axes=axes, grid=",".join(map(str, grid)), voxel=voxel,
                    offset=_log(rng, 1, 100000) if three else 0, pairing=pairing, dtype=dtype, layout=layout,
                    inverse=rng.random() < 0.5)
    Hk = rng.choice([1, 2, 5, 12])
    if op == "evict":
        Nk = _log(rng, 2, 40000)
        budget = rng.randint(1, Nk)
        sink = rng.randint(0, budget // 3)
        recent = rng.randint(0, budget // 3)
        lengths = ",".join(str(rng.randint(0, Nk)) for _ in range(B)) if rng.random() < 0.5 else ""
        return dict(op=op, B=B, Hk=Hk, d=d, Nk=Nk, budget=budget, sink=sink, recent=recent, lengths=lengths, layout=layout)
    rep = rng.choice([1, 1, 2, 3, 8])
    Nk = _log(rng, 1, 30000)
    most = 2_000_000_000 // (B * Hk * rep * Nk)
    Nq = 1 if rng.random() < 0.3 else max(1, min(_log(rng, 1, 16000), most))
    if op == "weights":
        lengths = ",".join(str(rng.randint(1, Nk)) for _ in range(B)) if rng.random() < 0.5 else ""
        return dict(op=op, B=B, H=Hk * rep, Hk=Hk, d=d, Nq=Nq, Nk=Nk, causal=0 if lengths else rng.choice([0, 1, 97]),
                    decay=rng.choice([0.0, 0.9, 1.0]), lengths=lengths, layout=layout)
    causal, cap, bias = rng.choice([0, 1, 97, 880]), rng.choice([0.0, 0.0, 30.0]), rng.random() < 0.3
    dq = dk = px = ""
    if rng.random() < 0.5:
        n = rng.randint(1, 9)
        rows = _docs(rng, B, Nk, n)
        dk = _text(rows)
        dq = _text(_docs(rng, B, Nq, n)) if Nq != Nk else dk
        if rng.random() < 0.5:
            px = ";".join(",".join(str(rng.randint(0, max(1, r[i + 1] - r[i]))) for i in range(n)) for r in rows)
    return dict(op=op, B=B, H=Hk * rep, Hk=Hk, d=d, Nq=Nq, Nk=Nk, causal=causal, cap=cap, bias=bias,
                docs_q=dq, docs_k=dk, prefix=px, layout=layout)


# ---------------------------------------------------------------- inputs

def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _rows(text, B):
    if not text:
        return None
    rows = [_ints(r) for r in text.split(";")]
    return rows * B if len(rows) == 1 else rows


def _table(rows):
    return None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")


def _normal(g, layout, B, H, N, d, dtype, scale=1.0, mean=None):
    """Random [B, H, N, d] values, head-major or as a view of token-major storage."""
    shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
    x = torch.randn(shape, generator=g, device="cuda") * scale
    if layout != "bhnd":
        x = x.transpose(1, 2)
    if mean is not None:
        x += mean
    return x.to(dtype)


def _blank(layout, B, H, N, d):
    shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return x if layout == "bhnd" else x.transpose(1, 2)


def _positions(grid, voxel, offset):
    """(t, h, w) of every token of a grid, in raster order or voxel by voxel (edge voxels clipped)."""
    T, Hh, W = grid
    t, h, w = torch.meshgrid(torch.arange(T), torch.arange(Hh), torch.arange(W), indexing="ij")
    p = torch.stack([t, h, w], -1).reshape(-1, 3)
    if voxel:
        vt, vh, vw = voxel
        key = ((p[:, 0] // vt) * 1000 + p[:, 1] // vh) * 1000 + p[:, 2] // vw
        p = p[torch.sort(key, stable=True).indices]
    p[:, 0] += offset
    return p


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, d, layout = c["B"], c["d"], c["layout"]
    if c["op"] == "rope":
        axes, grid, voxel = _ints(c["axes"]), _ints(c["grid"]), _ints(c["voxel"])
        dtype = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        if len(grid) == 3:
            c["pos"] = _positions(grid, voxel, c["offset"]).to("cuda", torch.int32)
            c["given"] = None
        else:  # explicit positions, as after an eviction
            N = grid[0]
            c["pos"] = torch.randint(0, 100000, (B, N, len(axes)), generator=g, device="cuda", dtype=torch.int32)
            c["given"] = c["pos"]
        N = math.prod(grid)
        c.update(axes=axes, grid=grid, voxel=voxel)
        c["q"] = _normal(g, layout, B, c["H"], N, d, dtype)
        c["k"] = _normal(g, layout, B, c["Hk"], N, d, dtype) if c["Hk"] else None
        return c
    Hk, Nk = c["Hk"], c["Nk"]
    if c["op"] == "evict":
        c["k"] = _normal(g, layout, B, Hk, Nk, d, torch.bfloat16)
        c["v"] = _normal(g, layout, B, Hk, Nk, d, torch.bfloat16)
        # accumulated weights are heavy-tailed, and whole runs of keys have the same small one
        w = torch.exp(2.0 * torch.randn(B, Hk, Nk, generator=g, device="cuda"))
        c["w"] = torch.where(w < 0.2, torch.full_like(w, 0.125), w)
        c["lengths"] = torch.tensor(_ints(c["lengths"]), dtype=torch.int32, device="cuda") if c["lengths"] else None
        m = c["budget"]
        c["out"] = (_blank(layout, B, Hk, m, d), _blank(layout, B, Hk, m, d),
                    torch.zeros(B, Hk, m, device="cuda"))
        return c
    H, Nq = c["H"], c["Nq"]
    mean = 0.5 * torch.randn(B, Hk, 1, d, generator=g, device="cuda")
    c["q"] = _normal(g, layout, B, H, Nq, d, torch.bfloat16, scale=1.4)
    c["k"] = _normal(g, layout, B, Hk, Nk, d, torch.bfloat16, mean=mean)
    if c["op"] == "weights":
        lens = _ints(c["lengths"]) or [Nk] * B
        c["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if c["lengths"] else None
        c["docs_q"] = c["docs_k"] = c["prefix"] = None
        if c["lengths"] is not None:
            c["docs_q"] = torch.tensor([[0, Nq]] * B, dtype=torch.int32, device="cuda")
            c["docs_k"] = torch.tensor([[0, n] for n in lens], dtype=torch.int32, device="cuda")
        c["cap"], c["slopes"] = 0.0, None
        c["lse"] = _log_sums(c)
        c["w"] = torch.exp(torch.randn(B, Hk, Nk, generator=g, device="cuda"))
        return c
    c["v"] = _normal(g, layout, B, Hk, Nk, d, torch.bfloat16)
    for name in ("docs_q", "docs_k", "prefix"):
        c[name] = _table(_rows(c[name], B))
    c["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H) if c["bias"] else None
    return c


# ---------------------------------------------------------------- plain forms

def _spans(c):
    """Per query row the half-open span of visible keys, its position and its document's first key: each [B, Nq]."""
    B, Nq, Nk = c["B"], c["Nq"], c["Nk"]
    i = torch.arange(Nq, device="cuda")
    if c["docs_k"] is None:
        qs, qe, ks, ke, px = 0 * i, 0 * i + Nq, 0 * i, 0 * i + Nk, 0 * i
        qs, qe, ks, ke, px = (x.expand(B, Nq) for x in (qs, qe, ks, ke, px))
    else:
        dq, dk = c["docs_q"].long(), c["docs_k"].long()
        n = dq.shape[1] - 1
        doc = (dq[:, None, 1:] <= i[None, :, None]).sum(-1)  # documents that end at or before row i
        at = doc.clamp(max=n - 1)
        pick = lambda t: torch.gather(t, 1, at)  # noqa: E731
        qs, qe, ks, ke = pick(dq[:, :-1]), pick(dq[:, 1:]), pick(dk[:, :-1]), pick(dk[:, 1:])
        ke = torch.where(doc < n, ke, ks)
        px = pick(c["prefix"].long()) if c["prefix"] is not None else 0 * ks
    n = ke - ks
    p = i - qs + n - (qe - qs)  # the rows of a document are its last positions
    hi = n
    if c["causal"]:
        f = c["causal"]
        hi = (torch.div(p, f, rounding_mode="floor") + 1) * f
        hi = torch.minimum(torch.maximum(torch.maximum(hi, px), 0 * hi), n)
    return ks, ks + hi, p, ks


def _scores(c, dtype):
    """Scaled, capped, biased and masked scores [B, Hk, R, Nq, Nk]."""
    B, H, Hk, Nq, Nk, d = c["B"], c["H"], c["Hk"], c["Nq"], c["Nk"], c["d"]
    R = H // Hk
    q = c["q"].to(dtype).reshape(B, Hk, R * Nq, d)
    s = torch.matmul(q, c["k"].to(dtype).transpose(-1, -2)).view(B, Hk, R, Nq, Nk).mul_(d ** -0.5)
    if c["cap"]:
        s.div_(c["cap"]).tanh_().mul_(c["cap"])
    lo, hi, p, first = _spans(c)
    j = torch.arange(Nk, device="cuda")
    if c["slopes"] is not None:
        far = (p[:, :, None] - (j - first[:, :, None])).abs().to(dtype)
        s.sub_(c["slopes"].to(dtype).view(1, Hk, R, 1, 1) * far[:, None, None])
    out = (j < lo[:, :, None]) | (j >= hi[:, :, None])
    return s.masked_fill_(out[:, None, None], -math.inf)


def _log_sums(c):
    s = _scores(c, torch.float32)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    return (s.sub_(m).exp_().sum(-1).log() + m[..., 0]).view(c["B"], c["H"], c["Nq"])


def _rope_plain(x, c, dtype):
    """x rotated by its positions' angles; the angles in 64 bits."""
    axes, d = c["axes"], c["d"]
    pos = c["pos"].double()
    if pos.dim() == 2:
        pos = pos[None]
    angle = torch.cat([pos[..., a:a + 1] * 10000.0 ** (-torch.arange(0, n, 2, device="cuda").double() / n)
                       for a, n in enumerate(axes)], -1)[:, None]  # [B or 1, 1, N, pairs]
    cos, sin = angle.cos().to(dtype), angle.sin().to(dtype)
    if c["inverse"]:
        sin = -sin
    r = sum(axes)
    y = x.to(dtype).clone()
    if c["pairing"] == "half":
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _attend_plain(c):
    B, H, Hk, Nq, d = c["B"], c["H"], c["Hk"], c["Nq"], c["d"]
    s = _scores(c, torch.float32)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, c["Nk"]), c["v"].float()).view(B, H, Nq, d)
    l = l.view(B, H, Nq, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.to(torch.bfloat16), (l.log() + m.view(B, H, Nq, 1))[..., 0]


def _weights_plain(c):
    B, Hk, Nq, Nk = c["B"], c["Hk"], c["Nq"], c["Nk"]
    s = _scores(c, torch.float32)
    lse = c["lse"].view(B, Hk, -1, Nq, 1)
    got = s.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_().sum((2, 3))
    out = got + c["decay"] * c["w"]
    if c["lengths"] is None:
        return out
    return torch.where(torch.arange(Nk, device="cuda") < c["lengths"].view(B, 1, 1), out, c["w"])


def _evict_plain(c):
    B, Hk, Nk, m = c["B"], c["Hk"], c["Nk"], c["budget"]
    n = torch.full((B,), Nk, device="cuda") if c["lengths"] is None else c["lengths"].long()
    n = n.view(B, 1, 1)
    j = torch.arange(Nk, device="cuda").expand(B, Hk, Nk)
    stays = (j < c["sink"]) | (j >= n - c["recent"])
    rank = torch.where(j >= n, 2, torch.where(stays, 0, 1))
    order = torch.sort(c["w"], dim=-1, descending=True, stable=True).indices
    order = torch.gather(order, 2, torch.sort(torch.gather(rank, 2, order), dim=-1, stable=True).indices)
    keep = n.clamp(max=m)
    top = order[:, :, :m]
    slot = torch.arange(m, device="cuda").expand(B, Hk, m)
    kept = torch.sort(torch.where(slot < keep, top, Nk), dim=-1).values
    live = kept < Nk
    at = torch.where(live, kept, 0)
    for to, of in zip(c["out"][:2], (c["k"], c["v"])):
        rows = torch.gather(of, 2, at[..., None].expand(B, Hk, m, c["d"]))
        to.copy_(torch.where(live[..., None], rows, to))
    w = c["out"][2]
    w.copy_(torch.where(live, torch.gather(c["w"], 2, at), w))
    return (torch.where(live, kept, -1).int(),) + c["out"]


def run(state):
    c = state
    if own:
        return _run_own(c)
    if c["op"] == "rope":
        y = [None if x is None else _rope_plain(x, c, torch.float32).to(x.dtype) for x in (c["q"], c["k"])]
        return [t for t in y if t is not None]
    return {"masked": _attend_plain, "weights": _weights_plain, "evict": _evict_plain}[c["op"]](c)


def _run_own(c):
    from video_dit_sparse_gb300 import binding as sa
    if c["op"] == "rope":
        if c["given"] is not None:
            y = sa.sparse_attn_rope(c["q"], c["k"], axes=c["axes"], positions=c["given"], pairing=c["pairing"],
                                    inverse=c["inverse"])
        else:
            y = sa.sparse_attn_rope(c["q"], c["k"], axes=c["axes"], grid=c["grid"], voxel=c["voxel"] or None,
                                    offset=(c["offset"], 0, 0), pairing=c["pairing"], inverse=c["inverse"])
        return [y] if c["k"] is None else list(y)
    if c["op"] == "masked":
        return sa.sparse_attn_forward_masked(c["q"], c["k"], c["v"], causal=c["causal"], cap=c["cap"], slopes=c["slopes"],
                                             docs_q=c["docs_q"], docs_k=c["docs_k"], prefix=c["prefix"])
    if c["op"] == "weights":
        return sa.sparse_attn_cache_weights(c["q"], c["k"], c["lse"], c["w"], decay=c["decay"], causal=c["causal"],
                                            lengths=c["lengths"])
    return sa.sparse_attn_cache_evict(c["w"], c["k"], c["v"], c["budget"], sink=c["sink"], recent=c["recent"],
                                      lengths=c["lengths"], out=c["out"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    def pairs_and_keys():
        """Visible (query, key) pairs of one head over the whole batch, and the keys that any row sees."""
        B, Nq, Nk, f = case["B"], case["Nq"], case["Nk"], case["causal"]
        if case["op"] == "weights":
            lens = _ints(case["lengths"]) or [Nk] * B
            dq, dk, px = [[0, Nq]] * B, [[0, n] for n in lens], None
        else:
            dq, dk, px = (_rows(case[x], B) for x in ("docs_q", "docs_k", "prefix"))
            if dk is None:
                dq, dk = [[0, Nq]] * B, [[0, Nk]] * B
        pairs = keys = 0
        for b in range(B):
            for e in range(len(dk[b]) - 1):
                nq, nk = dq[b][e + 1] - dq[b][e], dk[b][e + 1] - dk[b][e]
                pre = px[b][e] if px else 0
                top = 0
                for i in range(nq):
                    hi = nk
                    if f:
                        hi = max(0, min(nk, max(((i + nk - nq) // f + 1) * f, pre)))
                    pairs += hi
                    top = max(top, hi)
                keys += top
        return pairs, keys

    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        n = B * (case["H"] + case["Hk"]) * math.prod(_ints(case["grid"]))
        return {"bytes": 2 * n * d * (4 if case["dtype"] == "fp32" else 2), "flops": 3 * n * sum(_ints(case["axes"]))}
    if case["op"] == "evict":
        lens = _ints(case["lengths"]) or [case["Nk"]] * B
        kept = case["Hk"] * sum(min(n, case["budget"]) for n in lens)
        return {"bytes": case["Hk"] * sum(lens) * 4 + kept * (2 * 2 * d * 2 + 4 + 4), "flops": 0}
    pairs, keys = pairs_and_keys()
    H, Hk, Nq = case["H"], case["Hk"], case["Nq"]
    if case["op"] == "weights":
        return {"bytes": B * H * Nq * (2 * d + 4) + Hk * keys * (2 * d + 8), "flops": 2 * d * pairs * H}
    return {"bytes": B * H * Nq * (4 * d + 4) + Hk * keys * 4 * d, "flops": 4 * d * pairs * H}


# ---------------------------------------------------------------- 64-bit values

def exact(case, seed):
    c = prepare(case, seed)

    def rotated(x):
        pos = c["pos"].double()
        pos = pos[None] if pos.dim() == 2 else pos
        y = x.double().clone()
        first, r = 0, sum(c["axes"])
        for a, n in enumerate(c["axes"]):
            for i in range(n // 2):
                angle = pos[:, None, :, a] * math.pow(10000.0, -2.0 * i / n)
                if c["inverse"]:
                    angle = -angle
                e = first + i
                u, v = (e, e + r // 2) if c["pairing"] == "half" else (2 * e, 2 * e + 1)
                z = torch.complex(y[..., u], y[..., v]) * torch.polar(torch.ones_like(angle), angle)
                y[..., u], y[..., v] = z.real, z.imag
            first += n // 2
        return y

    def scores(b, h):
        """One head's 64-bit scores, the masked ones -inf, document by document."""
        Nq, Nk, f = c["Nq"], c["Nk"], c["causal"]
        s = torch.full((Nq, Nk), -math.inf, dtype=torch.float64, device="cuda")
        q, k = c["q"][b, h].double(), c["k"][b, h // (c["H"] // c["Hk"])].double()
        dq = [0, Nq] if c["docs_q"] is None else c["docs_q"][b].tolist()
        dk = [0, Nk] if c["docs_k"] is None else c["docs_k"][b].tolist()
        px = [0] * (len(dk) - 1) if c["prefix"] is None else c["prefix"][b].tolist()
        for e in range(len(dk) - 1):
            (q0, q1), (k0, k1) = dq[e:e + 2], dk[e:e + 2]
            if q1 <= q0 or k1 <= k0:
                continue
            x = q[q0:q1] @ k[k0:k1].T / math.sqrt(c["d"])
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            at = torch.arange(k1 - k0 - (q1 - q0), k1 - k0, device="cuda")[:, None]
            key = torch.arange(k1 - k0, device="cuda")[None]
            if c["slopes"] is not None:
                x = x - float(c["slopes"][h]) * (at - key).abs()
            if f:
                sees = (torch.div(key, f, rounding_mode="floor") <= torch.div(at, f, rounding_mode="floor")) | (key < px[e])
                x = torch.where(sees, x, torch.full_like(x, -math.inf))
            s[q0:q1, k0:k1] = x
        return s

    if c["op"] == "rope":
        return [rotated(x) for x in (c["q"], c["k"]) if x is not None]
    B, Hk, Nk = c["B"], c["Hk"], c["Nk"]
    if c["op"] == "evict":
        m, w, k, v = c["budget"], c["w"].cpu(), c["k"].cpu().double(), c["v"].cpu().double()
        outs = [torch.full((B, Hk, m), -1, dtype=torch.int32), torch.zeros(B, Hk, m, c["d"], dtype=torch.float64),
                torch.zeros(B, Hk, m, c["d"], dtype=torch.float64), torch.zeros(B, Hk, m, dtype=torch.float64)]
        for b in range(B):
            n = Nk if c["lengths"] is None else int(c["lengths"][b])
            for h in range(Hk):
                x = w[b, h, :n].tolist()
                fixed = [j for j in range(n) if j < c["sink"] or j >= n - c["recent"]] if n > m else list(range(n))
                have = set(fixed)
                rest = sorted((j for j in range(n) if j not in have), key=lambda j: (-x[j], j))
                kept = sorted(fixed + rest[:max(0, min(n, m) - len(fixed))])
                at = torch.tensor(kept, dtype=torch.long)
                for o, t in zip(outs, (at.int(), k[b, h, at], v[b, h, at], w[b, h, at].double())):
                    o[b, h, :len(kept)] = t
        return outs
    H, Nq, d = c["H"], c["Nq"], c["d"]
    if c["op"] == "weights":
        out = c["decay"] * c["w"].double()
        for b in range(B):
            for h in range(H):
                l = c["lse"][b, h].double()
                p = torch.exp(scores(b, h) - l[:, None])
                out[b, h // (H // Hk)] += torch.where(torch.isinf(l)[:, None], torch.zeros_like(p), p).sum(0)
            if c["lengths"] is not None:
                n = int(c["lengths"][b])
                out[b, :, n:] = c["w"][b, :, n:].double()
        return out
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, Nq, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            s = scores(b, h)
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(torch.isinf(lse[b, h]), torch.zeros_like(lse[b, h]), lse[b, h])[:, None])
            o[b, h] = p @ c["v"][b, h // (H // Hk)].double()
    return o, lse
