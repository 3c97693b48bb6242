"""Operators on both sides of the attention of a transformer with a rolling key-value cache, as cases that can be timed
and compared.

  norm_rope   every head's query and key normalised (root mean square, or mean and variance), scaled, and rotated by its
              position, in one pass
  gradient    the gradient of that: of the queries and keys, of the scales and shifts
  store       new keys and values into a cache held in 8 bits (e4m3) with a power-of-two scale for each head and block of
              tokens, and the cache's newest tokens read back
  attend      attention over such a cache: many query rows of a frame-causal chunk, or a new token or a few

`run` computes a case in plain tensor operations (own = False), or through the library's entry points (own = True).
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the 69K-token latent of a 720p clip, queries and keys of one layer in voxel order
        dict(name="norm_rope_video69k", op="norm_rope", B=1, H=24, Hk=24, d=128, axes="44,42,42", grid="18,48,80",
             voxel="2,8,8", offset=0, pairing="interleaved", dtype="bf16", layout="bhnd", norm="rms", weight="fp32"),
        # one chunk of 8 frames of 22x40 tokens entering a rolling window, straight from the projections (token-major),
        # normalised by mean and variance with a shift
        dict(name="norm_rope_chunk_layer", op="norm_rope", B=1, H=12, Hk=12, d=128, axes="44,42,42", grid="8,22,40",
             voxel="", offset=24, pairing="interleaved", dtype="bf16", layout="bnhd", norm="layer", weight="same"),
        # one new token of four sequences, shared key heads, explicit positions: latency
        dict(name="norm_rope_token", op="norm_rope", B=4, H=24, Hk=6, d=128, axes="128", grid="1", voxel="", offset=0,
             pairing="half", dtype="bf16", layout="bnhd", norm="rms", weight="same"),
        # a training step's gradient through 16K tokens of 24 heads
        dict(name="gradient_16k", op="gradient", B=1, H=24, Hk=24, d=128, axes="44,42,42", grid="16,32,32", voxel="2,8,8",
             offset=0, pairing="interleaved", dtype="bf16", layout="bnhd", norm="rms", weight="fp32"),
        # the same of a small model in fp32 with mean, variance and shift, an odd number of tokens: latency
        dict(name="gradient_layer_fp32", op="gradient", B=2, H=3, Hk=1, d=64, axes="32,32", grid="1237", voxel="", offset=0,
             pairing="half", dtype="fp32", layout="bhnd", norm="layer", weight="same"),
        # a chunk's keys and values appended behind a full window
        dict(name="store_chunk", op="store", B=1, Hk=12, d=128, N=35200, n=7040, block=128, start="28160", counts="",
             read=7040, layout="bnhd"),
        # one token of each of four sequences of different length, into blocks that hold earlier tokens
        dict(name="store_token", op="store", B=4, Hk=6, d=128, N=28160, n=1, block=64, start="28158,7040,19999,27998",
             counts="", read=64, layout="bhnd"),
        # a chunk's queries over the whole window; a frame sees itself and what came before
        dict(name="attend_frames", op="attend", B=1, H=12, Hk=12, d=128, Nq=7040, Nk=28160, causal=880, block=128,
             lengths="", layout="bhnd"),
        # shared key heads, token-causal, an odd length, small blocks
        dict(name="attend_shared", op="attend", B=2, H=16, Hk=4, d=64, Nq=4099, Nk=4099, causal=1, block=32, lengths="",
             layout="bnhd"),
        # one new token per sequence over caches of different fill, shared key heads
        dict(name="attend_token", op="attend", B=4, H=24, Hk=6, d=128, Nq=1, Nk=28160, causal=1, block=64,
             lengths="28160,7041,20000,27999", layout="bhnd"),
        # one new token over a long cache
        dict(name="attend_token_long", op="attend", B=1, H=32, Hk=8, d=128, Nq=1, Nk=262144, causal=0, block=128,
             lengths="", layout="bhnd"),
        # one new token over a single frame: latency
        dict(name="attend_token_frame", op="attend", B=1, H=12, Hk=12, d=128, Nq=1, Nk=880, causal=0, block=16, lengths="",
             layout="bhnd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(values):
    return ",".join(str(x) for x in values)


def draw(rng):
    op = rng.choice(["norm_rope", "gradient", "store", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    layout = rng.choice(["bhnd", "bnhd"])
    B = rng.choice([1, 1, 2, 3])
    if op in ("norm_rope", "gradient"):
        H = rng.choice([1, 3, 12, 24])
        Hk, dtype = rng.choice([0, 1, H]), rng.choice(["bf16", "bf16", "fp32"])
        three = rng.random() < 0.7
        if three:
            grid = [rng.randint(1, 12), rng.randint(1, 45), rng.randint(1, 80)]
            axes = {128: rng.choice(["44,42,42", "32,48,48"]), 64: "24,20,20"}[d]
            voxel = rng.choice(["", "2,8,8", "3,5,4"])
        else:
            grid, axes, voxel = [_log(rng, 1, 40000)], rng.choice(["%d" % d, "32,32", "16,24,24"]), ""
        most = 400_000_000 // (B * (H + Hk) * d * (4 if dtype == "fp32" else 2) * math.prod(grid[1:]))
        grid[0] = max(1, min(grid[0], most))
        return dict(op=op, B=B, H=H, Hk=Hk, d=d, axes=axes, grid=_text(grid), voxel=voxel,
                    offset=_log(rng, 1, 100000) if three else 0, pairing=rng.choice(["interleaved", "half"]), dtype=dtype,
                    layout=layout, norm=rng.choice(["rms", "rms", "layer"]), weight=rng.choice(["same", "fp32", ""]))
    block = rng.choice([16, 32, 64, 128])
    Hk = rng.choice([1, 2, 5, 12])
    if op == "store":
        N = _log(rng, 2, 40000)
        n = min(N, _log(rng, 1, 8000))
        start = [rng.randint(0, N - n) for _ in range(B)]
        counts = [rng.randint(0, n) for _ in range(B)] if rng.random() < 0.4 else []
        return dict(op=op, B=B, Hk=Hk, d=d, N=N, n=n, block=block, start=_text(start), counts=_text(counts),
                    read=rng.randint(1, N), layout=layout)
    R = rng.choice([1, 1, 2, 3, 4, 8])
    Nk = _log(rng, 1, 30000)
    most = max(1, 1_500_000_000 // (B * Hk * R * Nk))
    kind = rng.random()
    Nq = 1 if kind < 0.35 else rng.randint(2, 40) if kind < 0.6 else _log(rng, 1, 12000)
    lengths = [rng.randint(1, Nk) for _ in range(B)] if rng.random() < 0.5 else []
    return dict(op=op, B=B, H=Hk * R, Hk=Hk, d=d, Nq=max(1, min(Nq, most)), Nk=Nk, causal=rng.choice([0, 1, 97, 880]),
                block=block, lengths=_text(lengths), layout=layout)


# ---------------------------------------------------------------- inputs

def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _index(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(g, layout, B, H, N, d, dtype, scale=1.0, mean=None):
    """Random [B, H, N, d] values, head-major or as a view of token-major storage."""
    x = torch.randn((B, H, N, d) if layout == "bhnd" else (B, N, H, d), generator=g, device="cuda") * scale
    if layout != "bhnd":
        x = x.transpose(1, 2)
    if mean is not None:
        x += mean
    return x.to(dtype)


def _positions(grid, voxel, offset):
    """(t, h, w) of every token of a grid, in raster order or voxel by voxel (edge voxels clipped)."""
    t, h, w = torch.meshgrid(*(torch.arange(n) for n in grid), indexing="ij")
    p = torch.stack([t, h, w], -1).reshape(-1, 3)
    if voxel:
        key = ((p[:, 0] // voxel[0]) * 1000 + p[:, 1] // voxel[1]) * 1000 + p[:, 2] // voxel[2]
        p = p[torch.sort(key, stable=True).indices]
    p[:, 0] += offset
    return p


def _scale(top):
    """The least power of two that brings values up to `top` to e4m3's largest, 448 = 0.875 2^9, or below (0 for 0)."""
    m, e = torch.frexp(top)
    bits = (e + (m > 0.875).int() - 9 + 127) << 23  # (a power computed in floating point may be a step off)
    return torch.where(top > 0, bits.view(torch.float32), 0.0)


def _held(x, block):
    """What a cache filled with x [B, H, N, d] holds: e4m3 codes (of x's layout), and the scales [B, H, blocks]."""
    N = x.shape[2]
    blocks = -(-N // block)
    top = torch.zeros(x.shape[:2] + (blocks * block,), device="cuda")
    top[:, :, :N] = x.abs().amax(-1)
    top = top.view(x.shape[:2] + (blocks, block)).amax(-1)
    scale = _scale(top)
    per = scale.repeat_interleave(block, -1)[:, :, :N, None]
    return (x / torch.where(per > 0, per, 1.0)).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, d, layout = c["B"], c["d"], c["layout"]
    if c["op"] in ("norm_rope", "gradient"):
        axes, grid, voxel = _ints(c["axes"]), _ints(c["grid"]), _ints(c["voxel"])
        dtype = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        N = math.prod(grid)
        if len(grid) == 3:
            c["pos"] = _positions(grid, voxel, c["offset"]).to("cuda", torch.int32)
            c["given"] = None
        else:  # explicit positions, as after an eviction
            c["pos"] = torch.randint(0, 100000, (B, N, len(axes)), generator=g, device="cuda", dtype=torch.int32)
            c["given"] = c["pos"]
        c.update(axes=axes, grid=grid, voxel=voxel)
        for name, H in (("q", c["H"]), ("k", c["Hk"])):
            c[name] = c["d" + name] = c[name + "w"] = c[name + "b"] = None
            if not H:
                continue
            # what a projection gives: heads and channels of different size, off centre
            spread = torch.exp(0.5 * torch.randn(1, H, 1, d, generator=g, device="cuda"))
            off = 0.3 * torch.randn(1, H, 1, d, generator=g, device="cuda")
            c[name] = _normal(g, layout, B, H, N, d, dtype, scale=1.0, mean=off)
            c[name] = (c[name] * spread).to(dtype)
            if c["weight"]:
                kind = torch.float32 if c["weight"] == "fp32" else dtype
                c[name + "w"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(kind)
                if c["norm"] == "layer":
                    c[name + "b"] = (0.2 * torch.randn(d, generator=g, device="cuda")).to(kind)
            if c["op"] == "gradient":
                c["d" + name] = _normal(g, layout, B, H, N, d, dtype, scale=0.1)
        return c
    Hk, block = c["Hk"], c["block"]
    N = c["N"] if c["op"] == "store" else c["Nk"]
    mean = 0.5 * torch.randn(B, Hk, 1, d, generator=g, device="cuda")
    loud = torch.exp(0.7 * torch.randn(B, Hk, N, 1, generator=g, device="cuda"))  # tokens of different size
    c["k8"], c["ks"] = _held(_normal(g, layout, B, Hk, N, d, torch.float32, mean=mean), block)
    c["v8"], c["vs"] = _held(_normal(g, layout, B, Hk, N, d, torch.float32) * loud, block)
    if c["op"] == "store":
        n, start, counts = c["n"], _ints(c["start"]), _ints(c["counts"])
        c["k"] = _normal(g, layout, B, Hk, n, d, torch.bfloat16, mean=mean)
        c["v"] = _normal(g, layout, B, Hk, n, d, torch.bfloat16) * torch.exp(
            torch.randn(B, Hk, n, 1, generator=g, device="cuda")).bfloat16()
        ends = [s + (counts[b] if counts else n) for b, s in enumerate(start)]
        c["first"] = _index([max(0, e - c["read"]) for e in ends])
        c["start"], c["counts"] = _index(start), _index(counts) if counts else None
        return c
    H, Nq = c["H"], c["Nq"]
    c["q"] = _normal(g, layout, B, H, Nq, d, torch.bfloat16, scale=1.4)
    c["lengths"] = _index(_ints(c["lengths"])) if c["lengths"] else None
    c["out"] = torch.empty_like(c["q"])  # a serving program keeps its output buffers
    c["lse"] = torch.empty(B, H, Nq, device="cuda")
    return c


# ---------------------------------------------------------------- plain forms

def _turns(c, dtype):
    """cos and sin [B or 1, 1, N, pairs] of the positions' angles; the angles in 64 bits."""
    pos = c["pos"].double()
    pos = pos[None] if pos.dim() == 2 else pos
    angle = torch.cat([pos[..., a:a + 1] * 10000.0 ** (-torch.arange(0, n, 2, device="cuda").double() / n)
                       for a, n in enumerate(c["axes"])], -1)[:, None]
    return angle.cos().to(dtype), angle.sin().to(dtype)


def _turned(y, c, back=False):
    """y rotated by its positions' angles, or back."""
    cos, sin = _turns(c, y.dtype)
    sin = -sin if back else sin
    r = sum(c["axes"])
    y = y.clone()
    one, two = (slice(0, r // 2), slice(r // 2, r)) if c["pairing"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = a * cos - b * sin, a * sin + b * cos
    return y


def _normalised(x, c):
    """(x - mean) / deviation and 1 / deviation, over the last axis."""
    x = x.float()
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _norm_rope_plain(c):
    out = []
    for name in ("q", "k"):
        if c[name] is None:
            continue
        y = _normalised(c[name], c)[0]
        if c[name + "w"] is not None:
            y = y * c[name + "w"].float()
        if c[name + "b"] is not None:
            y = y + c[name + "b"].float()
        out.append(_turned(y, c).to(c[name].dtype))
    return out


def _gradient_plain(c):
    out = []
    for name in ("q", "k"):
        if c[name] is None:
            continue
        n, r = _normalised(c[name], c)
        g = _turned(c["d" + name].float(), c, back=True)
        h = g if c[name + "w"] is None else g * c[name + "w"].float()
        dx = h - n * (h * n).mean(-1, keepdim=True)
        if c["norm"] == "layer":
            dx = dx - h.mean(-1, keepdim=True)
        dw = None if c[name + "w"] is None else (g * n).sum((0, 1, 2))
        db = None if c[name + "b"] is None else g.sum((0, 1, 2))
        out += [t for t in ((dx * r).to(c[name].dtype), dw, db) if t is not None]
    return out


def _store_plain(c):
    """Whole blocks of the cache are taken out, changed and put back."""
    B, Hk, d, N, n, block = c["B"], c["Hk"], c["d"], c["N"], c["n"], c["block"]
    count = torch.full((B,), n, device="cuda") if c["counts"] is None else c["counts"].long()
    start = c["start"].long()
    nb = min((n - 1) // block + 2, -(-N // block))
    at = (start // block)[:, None] + torch.arange(nb, device="cuda")  # blocks [B, nb]
    at = torch.minimum(at, torch.full_like(at, -(-N // block) - 1))  # (past the last one: that one again)
    token = (at[:, :, None] * block + torch.arange(block, device="cuda")).view(B, 1, nb * block)
    inside = token < N
    put = inside & (token >= start.view(B, 1, 1)) & (token < (start + count).view(B, 1, 1))
    pick = (token - start.view(B, 1, 1)).clamp(0, n - 1)
    rows = token.clamp(max=N - 1).expand(B, Hk, -1)[..., None].expand(-1, -1, -1, d)
    of = at[:, None].expand(B, Hk, nb)
    for codes, scales, new in ((c["k8"], c["ks"], c["k"]), (c["v8"], c["vs"], c["v"])):
        had = torch.gather(scales, 2, of)
        old = torch.gather(codes.view(torch.uint8), 2, rows).view(torch.float8_e4m3fn).float()
        old = old * had.repeat_interleave(block, -1)[..., None]
        x = torch.gather(new.float(), 2, pick.expand(B, Hk, -1)[..., None].expand(-1, -1, -1, d))
        x = torch.where(put[..., None], x, torch.where(inside[..., None], old, 0.0))
        top = torch.where(put[..., None], x.abs(), 0.0).amax(-1).view(B, Hk, nb, block).amax(-1)
        want = _scale(top)
        whole = (put | ~inside).view(B, 1, nb, block).all(-1)
        some = put.view(B, 1, nb, block).any(-1)
        scale = torch.where(whole & some, want, torch.maximum(want, had))
        per = scale.repeat_interleave(block, -1)[..., None]
        made = (x / torch.where(per > 0, per, 1.0)).to(torch.float8_e4m3fn).view(torch.uint8)
        made = torch.where(inside[..., None] & some.repeat_interleave(block, -1)[..., None], made,
                           torch.gather(codes.view(torch.uint8), 2, rows))
        end = (N - 1 - start // block * block).clamp(max=nb * block - 1)  # (rows past the cache's end: its last row again)
        last = torch.gather(made, 2, end.view(B, 1, 1, 1).expand(B, Hk, 1, d))
        codes.view(torch.uint8).scatter_(2, rows, torch.where(inside[..., None], made, last))
        scales.scatter_(2, of, scale)
    where = c["first"].long().view(B, 1, 1) + torch.arange(c["read"], device="cuda")
    there = where < N
    where = where.clamp(max=N - 1).expand(B, Hk, -1)
    out = []
    for codes, scales in ((c["k8"], c["ks"]), (c["v8"], c["vs"])):
        x = torch.gather(codes.view(torch.uint8), 2, where[..., None].expand(-1, -1, -1, d)).view(torch.float8_e4m3fn)
        x = x.float() * torch.gather(scales, 2, where // block)[..., None]
        out.append(torch.where(there[..., None], x, 0.0).to(torch.bfloat16))
    return out + [c["ks"], c["vs"]]


def _sees(c):
    """Per query row the number of keys that it sees [B, Nq]: the rows are a sequence's last positions."""
    B, Nq, Nk, f = c["B"], c["Nq"], c["Nk"], c["causal"]
    n = torch.full((B,), Nk, device="cuda") if c["lengths"] is None else c["lengths"].long()
    n = n[:, None].expand(B, Nq)
    if not f:
        return n
    p = n - Nq + torch.arange(Nq, device="cuda")
    end = (torch.div(p, f, rounding_mode="floor") + 1) * f
    return torch.minimum(end.clamp(min=0), n)


def _attend_plain(c):
    B, H, Hk, Nq, Nk, d, block = c["B"], c["H"], c["Hk"], c["Nq"], c["Nk"], c["d"], c["block"]
    R = H // Hk

    def values(codes, scales):
        return codes.float() * scales.repeat_interleave(block, -1)[:, :, :Nk, None]

    q = c["q"].float().reshape(B, Hk, R * Nq, d)
    s = torch.matmul(q, values(c["k8"], c["ks"]).transpose(-1, -2)).view(B, Hk, R, Nq, Nk).mul_(d ** -0.5)
    out = torch.arange(Nk, device="cuda") >= _sees(c)[:, :, None]
    s = s.masked_fill_(out[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, Nk), values(c["v8"], c["vs"])).view(B, H, Nq, d)
    l = l.view(B, H, Nq, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.to(torch.bfloat16), (l.log() + m.view(B, H, Nq, 1))[..., 0]


def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _norm_rope_plain, "gradient": _gradient_plain, "store": _store_plain,
            "attend": _attend_plain}[state["op"]](state)


def _run_own(c):
    from video_dit_sparse_gb300 import binding as sa
    if c["op"] in ("norm_rope", "gradient"):
        if c["given"] is not None:
            where = dict(positions=c["given"])
        else:
            where = dict(grid=c["grid"], voxel=c["voxel"] or None, offset=(c["offset"], 0, 0))
        if c["op"] == "norm_rope":
            y = sa.sparse_attn_norm_rope(c["q"], c["k"], norm=c["norm"], q_weight=c["qw"], k_weight=c["kw"], q_bias=c["qb"],
                                         k_bias=c["kb"], eps=1e-6, axes=c["axes"], pairing=c["pairing"], **where)
            return [y] if c["k"] is None else list(y)
        made = sa.sparse_attn_norm_rope_backward(c["dq"], c["dk"], c["q"], c["k"], norm=c["norm"], q_weight=c["qw"],
                                                 k_weight=c["kw"], q_bias=c["qb"], k_bias=c["kb"], eps=1e-6, axes=c["axes"],
                                                 pairing=c["pairing"], **where)
        return [t for t in made if t is not None]
    cache = sa.Cache8(c["k8"], c["v8"], c["ks"], c["vs"], c["block"])
    if c["op"] == "store":
        sa.sparse_attn_cache8_append(cache, c["k"], c["v"], c["start"], counts=c["counts"])
        k, v = sa.sparse_attn_cache8_read(cache, c["first"], c["read"])
        return [k, v, c["ks"], c["vs"]]
    return sa.sparse_attn_forward_cache8(c["q"], cache, causal=c["causal"], lengths=c["lengths"], out=c["out"], lse=c["lse"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, d = case["B"], case["d"]
    if case["op"] in ("norm_rope", "gradient"):
        n = B * (case["H"] + case["Hk"]) * math.prod(_ints(case["grid"]))
        size = 4 if case["dtype"] == "fp32" else 2
        if case["op"] == "norm_rope":
            return {"bytes": 2 * n * d * size, "flops": 7 * n * d}
        return {"bytes": 3 * n * d * size, "flops": 14 * n * d}
    Hk, block = case["Hk"], case["block"]
    if case["op"] == "store":
        counts = _ints(case["counts"]) or [case["n"]] * B
        rows, back = Hk * sum(counts), Hk * B * min(case["read"], case["N"])
        scales = sum(-(-x // block) for x in counts) * Hk
        return {"bytes": rows * d * (2 + 1) * 2 + back * d * (1 + 2) * 2 + scales * 8, "flops": 2 * rows * d}
    H, Nq, Nk, f = case["H"], case["Nq"], case["Nk"], case["causal"]
    pairs = keys = 0
    for n in _ints(case["lengths"]) or [Nk] * B:
        top = 0
        for i in range(Nq):
            hi = n if not f else max(0, min(n, ((i + n - Nq) // f + 1) * f))
            pairs += hi
            top = max(top, hi)
        keys += top
    return {"bytes": B * H * Nq * (4 * d + 4) + Hk * keys * 2 * d + Hk * -(-keys // block) * 8, "flops": 4 * d * pairs * H}


# ---------------------------------------------------------------- 64-bit values

def exact(case, seed):
    c = prepare(case, seed)
    B, d = c["B"], c["d"]

    def pairs():
        """(first element, second element, angles [B or 1, 1, N]) of every rotated pair."""
        pos = c["pos"].double()
        pos = pos[None] if pos.dim() == 2 else pos
        first, r = 0, sum(c["axes"])
        for a, n in enumerate(c["axes"]):
            for i in range(n // 2):
                e = first + i
                u, v = (e, e + r // 2) if c["pairing"] == "half" else (2 * e, 2 * e + 1)
                yield u, v, pos[:, None, :, a] * math.pow(10000.0, -2.0 * i / n)
            first += n // 2

    def spun(y, way):
        for u, v, angle in pairs():
            z = torch.complex(y[..., u], y[..., v]) * torch.polar(torch.ones_like(angle), way * angle)
            y[..., u], y[..., v] = z.real, z.imag
        return y

    if c["op"] in ("norm_rope", "gradient"):
        out = []
        for name in ("q", "k"):
            if c[name] is None:
                continue
            w = torch.ones(d, dtype=torch.float64, device="cuda") if c[name + "w"] is None else c[name + "w"].double()
            b = 0.0 if c[name + "b"] is None else c[name + "b"].double()
            x = c[name].double()
            mu = x.sum(-1, keepdim=True) / d if c["norm"] == "layer" else 0.0
            dev = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / d + 1e-6)
            if c["op"] == "norm_rope":
                out.append(spun((x - mu) / dev * w + b, 1.0))
                continue
            g = spun(c["d" + name].double(), -1.0)
            # y_j = w_j (x_j - mu) / dev: d y_j / d x_i = w_j (delta_ij - 1/d [layer] - n_i n_j / d) / dev
            n, h = (x - mu) / dev, g * w
            dot = torch.einsum("bhnd,bhnd->bhn", h, n)[..., None] / d
            mean = h.sum(-1, keepdim=True) / d if c["norm"] == "layer" else 0.0
            out.append((h - mean - n * dot) / dev)
            if c[name + "w"] is not None:
                out.append(torch.einsum("bhnd,bhnd->d", g, n))
            if c[name + "b"] is not None:
                out.append(torch.einsum("bhnd->d", g))
        return out
    def power(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    def binade(y):
        """The whole e with 2^e <= y < 2^(e + 1)."""
        e = torch.floor(torch.log2(y.clamp(min=1e-300)))
        return e - (power(e) > y).double() + (power(e + 1) <= y).double()

    if c["op"] == "store":
        N, n, block, Hk = c["N"], c["n"], c["block"], c["Hk"]
        outs, scales_out = [], []
        for codes, scales, new in ((c["k8"], c["ks"], c["k"]), (c["v8"], c["vs"], c["v"])):
            per = scales.double().repeat_interleave(block, -1)[:, :, :N, None]
            x, s = codes.double() * per, scales.double().clone()
            for b in range(B):
                i0 = int(c["start"][b])
                i1 = i0 + (n if c["counts"] is None else int(c["counts"][b]))
                if i1 <= i0:
                    continue
                x[b, :, i0:i1] = new[b, :, :i1 - i0].double()
                for j in range(i0 // block, (i1 - 1) // block + 1):
                    t0, t1 = j * block, min(N, (j + 1) * block)
                    fresh = x[b, :, max(t0, i0):min(t1, i1)].abs().amax((-1, -2))
                    # the least power of two that brings the largest value to 448 or below
                    low = power(binade(fresh / 448))
                    want = torch.where(fresh > 0, torch.where(low * 448 < fresh, 2 * low, low), 0.0)
                    s[b, :, j] = want if i0 <= t0 and t1 <= i1 else torch.maximum(want, s[b, :, j])
                    # to the nearest of e4m3's values, ties to even: steps of 2^-3 of the binade, 2^-9 at least
                    y = x[b, :, t0:t1] / torch.where(s[b, :, j] > 0, s[b, :, j], 1.0)[:, None, None]
                    step = power(binade(y.abs()).clamp(min=-6)) / 8
                    x[b, :, t0:t1] = torch.round(y / step) * step * s[b, :, j][:, None, None]
            back = torch.zeros(B, Hk, c["read"], d, dtype=torch.float64, device="cuda")
            for b in range(B):
                i0 = int(c["first"][b])
                part = x[b, :, i0:i0 + c["read"]]
                back[b, :, :part.shape[1]] = part
            outs.append(back)
            scales_out.append(s)
        return outs + scales_out
    H, Hk, Nq, Nk = c["H"], c["Hk"], c["Nq"], c["Nk"]
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    key = torch.arange(Nk, device="cuda")
    for b in range(B):
        n = Nk if c["lengths"] is None else int(c["lengths"][b])
        at = torch.arange(n - Nq, n, device="cuda")[:, None]
        sees = key[None] < n
        if c["causal"]:
            sees = sees & (torch.div(key[None], c["causal"], rounding_mode="floor")
                           <= torch.div(at, c["causal"], rounding_mode="floor"))
        for h in range(H):
            hk = h // (H // Hk)
            k = c["k8"][b, hk].double() * c["ks"][b, hk].double()[key // c["block"]][:, None]
            v = c["v8"][b, hk].double() * c["vs"][b, hk].double()[key // c["block"]][:, None]
            x = (c["q"][b, h].double() @ k.T / math.sqrt(d)).masked_fill(~sees, -math.inf)
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(lse[b, h]), torch.zeros_like(lse[b, h]), lse[b, h])[:, None])
            o[b, h] = p @ v
    return o, lse
