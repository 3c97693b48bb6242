"""GPU checks of the normalised rotation and its gradient against the 64-bit forms.

Tolerances.  fp32 sums over a row of d <= 128 values run through chains of at most 32 additions: off by 2^-19 of the
terms' magnitudes.  So n is off by at most T = 2^-18 (|n| + r mean |x|) (the mean that is taken off, then 1 / sqrt of
the squares' sum), y = R(n w + b) by the pair's |w| T + 2^-20 |n w + b| (the rotation's bound), and one rounding to
the output type.  The gradient: g is off by G = 2^-20 (|dy| of the pair), and dx, dw, db follow term by term below; sums
over rows run through chains of less than 512 additions (2^-15 of the terms' magnitudes)."""
import numpy as np
import pytest
import torch

from oracle import cache8_ops as P
from oracle import cache_ops as O

pytestmark = pytest.mark.gpu


def make(shape, dtype, seed, layout="bhnd", off=0.0, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    B, H, N, d = shape
    x = (torch.randn((B, H, N, d) if layout == "bhnd" else (B, N, H, d), generator=g) * sigma + off).to(dtype).cuda()
    return x if layout == "bhnd" else x.transpose(1, 2)


def vector(d, dtype, seed, mean=1.0):
    return (mean + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def pairs(m, axes, half):
    """Each value's own magnitude plus its partner's."""
    out, r = m.copy(), sum(axes)
    if half:
        out[..., :r // 2] = out[..., r // 2:r] = m[..., :r // 2] + m[..., r // 2:r]
    else:
        out[..., 0:r:2] = out[..., 1:r:2] = m[..., 0:r:2] + m[..., 1:r:2]
    return out


def n_error(x, n, r):
    return 2.0 ** -18 * (np.abs(n) + r * np.abs(x).mean(-1, keepdims=True))


def check(got, x, pos, axes, half, layer, eps, w, b, **rope):
    x64, w64, b64 = np64(x), np64(w), np64(b)
    want = P.norm_rope(x64, pos, axes, layer, eps, w64, b64, half=half, **rope)
    n, r = P.normalised(x64, layer, eps)
    y = np.abs(n * (1.0 if w is None else w64)) + (0.0 if b is None else np.abs(b64))
    off = n_error(x64, n, r) * (1.0 if w is None else np.abs(w64)) + 2.0 ** -20 * y
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) * (1 + 2.0 ** -8) + pairs(off, axes, half)
    err = np.abs(np64(got) - want)
    assert (err <= tol).all(), float((err - tol).max())


def check_grad(made, dy, x, pos, axes, half, layer, eps, w, b, **rope):
    dx, dw, db = made
    x64, g64, w64 = np64(x), np64(dy), np64(w)
    want, wantw, wantb = P.norm_rope_grad(g64, x64, pos, axes, layer, eps, w64, half=half, **rope)
    n, r = P.normalised(x64, layer, eps)
    t = n_error(x64, n, r)
    g = O.rope(g64, pos, axes, half=half, inverse=True, **rope)
    eg = 2.0 ** -20 * pairs(np.abs(g64), axes, half)
    aw = 1.0 if w is None else np.abs(w64)
    h, eh = np.abs(g) * aw, eg * aw + 2.0 ** -23 * np.abs(g) * aw
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    tol = eh + np.abs(n) * mean(eh * np.abs(n) + h * t) + t * mean(h * np.abs(n)) + mean(eh)
    tol = r * (tol + 2.0 ** -18 * (h + np.abs(n) * mean(h * np.abs(n)) + mean(h)))
    # (1 / deviation's own error, on the whole)
    tol = 1.01 * tol + (2.0 ** -18 + torch.finfo(x.dtype).eps / 2) * np.abs(want)
    err = np.abs(np64(dx) - want)
    assert (err <= tol).all(), float((err - tol).max())
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    if w is not None:
        tol = (eg * np.abs(n) + np.abs(g) * t + 2.0 ** -15 * np.abs(g * n)).sum((0, 1, 2))
        assert (np.abs(np64(dw) - wantw) <= tol).all(), float((np.abs(np64(dw) - wantw) - tol).max())
    if b is not None:
        tol = (eg + 2.0 ** -15 * np.abs(g)).sum((0, 1, 2))
        assert (np.abs(np64(db) - wantb) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("d,axes", [(128, (44, 42, 42)), (64, (24, 20, 20)), (64, (16, 8, 8)), (128, (2, 0, 14))])
@pytest.mark.parametrize("grid,voxel,layout", [((3, 5, 7), None, "bhnd"), ((5, 7, 9), (2, 3, 4), "bnhd"),
                                               ((1, 1, 1), (2, 8, 8), "bhnd")])
def test_grid(dtype, half, norm, d, axes, grid, voxel, layout):
    from video_dit_sparse_gb300 import binding as sa
    N = grid[0] * grid[1] * grid[2]
    q, k = make((2, 5, N, d), dtype, 1, layout, off=0.7), make((2, 2, N, d), dtype, 2, layout, off=-2.0)
    dq, dk = make((2, 5, N, d), dtype, 3, layout), make((2, 2, N, d), dtype, 4, layout)
    kind = dtype if d == 64 else torch.float32
    qw, kw, qb = vector(d, kind, 5), vector(d, kind, 6), vector(d, kind, 7, 0.0)
    off = (1000003, -7, 12)
    pairing = "half" if half else "interleaved"
    opt = dict(norm=norm, q_weight=qw, k_weight=kw, q_bias=qb, eps=1e-5, axes=axes, grid=grid, voxel=voxel, offset=off,
               pairing=pairing)
    y, z = sa.sparse_attn_norm_rope(q, k, **opt)
    pos = O.voxel_positions(grid, voxel, off)
    layer = norm == "layer"
    check(y, q, pos, axes, half, layer, 1e-5, qw, qb)
    check(z, k, pos, axes, half, layer, 1e-5, kw, None)
    made = sa.sparse_attn_norm_rope_backward(dq, dk, q, k, **opt)
    check_grad(made[:3], dq, q, pos, axes, half, layer, 1e-5, qw, qb)
    check_grad(made[3:], dk, k, pos, axes, half, layer, 1e-5, kw, None)


@pytest.mark.parametrize("N", [1, 31, 33, 257, 1200])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_positions_alone_and_without_vectors(N, norm):
    from video_dit_sparse_gb300 import binding as sa
    x, g = make((3, 4, N, 64), torch.float32, 5, off=3.0), make((3, 4, N, 64), torch.float32, 6)
    pos = np.random.default_rng(N).integers(-1000, 1000, size=(3, N, 2))
    opt = dict(norm=norm, axes=(16, 16), pairing="half", positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    check(sa.sparse_attn_norm_rope(x, **opt), x, pos, (16, 16), True, norm == "layer", 1e-6, None, None)
    made = sa.sparse_attn_norm_rope_backward(g, None, x, **opt)
    check_grad(made, g, x, pos, (16, 16), True, norm == "layer", 1e-6, None, None)


def test_rows_far_off_centre_zeros_and_what_is_not_finite():
    """A mean of a thousand deviations is taken off before the squares; a row of zeros gives the shift; NaN stays in its row."""
    from video_dit_sparse_gb300 import binding as sa
    opt = dict(axes=(64,), positions=torch.zeros(9, 1, dtype=torch.int32, device="cuda"))
    x = make((1, 2, 9, 64), torch.float32, 1, off=1000.0)
    b = vector(64, torch.float32, 3, 0.0)
    pos = np.zeros((9, 1), dtype=np.int64)
    check(sa.sparse_attn_norm_rope(x, norm="layer", q_bias=b, **opt), x, pos, (64,), False, True, 1e-6, None, b)
    for norm in ("rms", "layer"):
        y = make((1, 2, 9, 64), torch.float32, 2)
        y[0, 1, 3] = 0.0
        y[0, 0, 5, 7] = float("nan")
        y[0, 0, 6, 7] = float("inf")
        z = sa.sparse_attn_norm_rope(y, norm=norm, q_bias=b, eps=1e-6, **opt)
        assert torch.equal(z[0, 1, 3], b)
        bad = ~torch.isfinite(z).all(-1)
        assert bad[0, 0, 5] and bad[0, 0, 6] and int(bad.sum()) == 2
        g = make((1, 2, 9, 64), torch.float32, 4)
        dx, _, db = sa.sparse_attn_norm_rope_backward(g, None, y, norm=norm, q_bias=b, eps=1e-6, **opt)
        bad = ~torch.isfinite(dx).all(-1)
        assert bad[0, 0, 5] and bad[0, 0, 6] and int(bad.sum()) == 2
        assert torch.isfinite(db).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_gradient_matches_differences(norm):
    """<dy, y(x + t e) - y(x - t e)> / 2t = <dx, e> + <dw, e_w> + <db, e_b> for directions e."""
    from video_dit_sparse_gb300 import binding as sa
    kw = dict(norm=norm, axes=(24, 20, 20), grid=(2, 3, 5), offset=(9, 0, 0))
    x, g = make((1, 2, 30, 64), torch.float32, 3, off=0.4), make((1, 2, 30, 64), torch.float32, 4)
    w, b = vector(64, torch.float32, 8), vector(64, torch.float32, 9, 0.0)
    dx, dw, db = sa.sparse_attn_norm_rope_backward(g, None, x, q_weight=w, q_bias=b, **kw)
    t = 2.0 ** -6
    for seed in range(4):
        e, ew, eb = make((1, 2, 30, 64), torch.float32, 10 + seed), vector(64, torch.float32, 20 + seed, 0.0), vector(
            64, torch.float32, 30 + seed, 0.0)
        up = sa.sparse_attn_norm_rope(x + t * e, q_weight=w + t * ew, q_bias=b + t * eb, **kw).double()
        down = sa.sparse_attn_norm_rope(x - t * e, q_weight=w - t * ew, q_bias=b - t * eb, **kw).double()
        lhs = float((g.double() * (up - down)).sum() / (2 * t))
        rhs = float((dx.double() * e.double()).sum() + (dw.double() * ew.double()).sum() + (db.double() * eb.double()).sum())
        # 3840 terms |g| (|y''' e^3| t^2 / 6 + 2^-18 |y| / t), |y''' e^3| below 40 on average (|e| of a row is its |x|)
        # and |g| near 1, adding up at random: 5 sqrt(3840) of one term
        assert abs(lhs - rhs) <= 5 * 3840 ** 0.5 * (40 * t * t / 6 + 2.0 ** -18 * 3 / t)


def test_in_place_views_streams_and_repeats():
    from video_dit_sparse_gb300 import binding as sa
    B, H, Hk, N, d = 2, 6, 2, 77, 128
    buf = make((B, N, H + 2 * Hk, d), torch.bfloat16, 1)  # a fused projection, token-major
    q, k = buf[:, :, :H].transpose(1, 2), buf[:, :, H:H + Hk].transpose(1, 2)
    v = buf[:, :, H + Hk:].clone()
    w = vector(d, torch.float32, 2)
    opt = dict(axes=(128,), positions=torch.arange(N, dtype=torch.int32, device="cuda")[:, None], q_weight=w, k_weight=w)
    y, z = sa.sparse_attn_norm_rope(q, k, **opt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, z2 = sa.sparse_attn_norm_rope(q, k, stream=side, **opt)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(z, z2)
    g = make((B, H, N, d), torch.bfloat16, 3)
    one = sa.sparse_attn_norm_rope_backward(g, None, q, axes=(128,), positions=opt["positions"], q_weight=w)
    in_dy = g.clone()
    two = sa.sparse_attn_norm_rope_backward(in_dy, None, q, axes=(128,), positions=opt["positions"], q_weight=w, out=in_dy)
    assert two[0] is in_dy and torch.equal(one[0], in_dy) and torch.equal(one[1], two[1])
    wide = make((B, 1, N, d), torch.bfloat16, 4).expand(B, H, N, d)  # one head repeated
    assert torch.equal(sa.sparse_attn_norm_rope(wide, axes=(128,), positions=opt["positions"], out=torch.empty_like(g)),
                       sa.sparse_attn_norm_rope(wide.contiguous(), axes=(128,), positions=opt["positions"]))
    a, b = sa.sparse_attn_norm_rope(q, k, out=(q, k), **opt)
    assert a is q and torch.equal(q, y) and torch.equal(k, z) and torch.equal(buf[:, :, H + Hk:], v)


def test_graph_replays_and_sums_repeat():
    from video_dit_sparse_gb300 import binding as sa
    x, g = make((1, 24, 4099, 128), torch.bfloat16, 1), make((1, 24, 4099, 128), torch.bfloat16, 2)
    w = vector(128, torch.bfloat16, 3)
    opt = dict(axes=(44, 42, 42), positions=torch.arange(4099 * 3, dtype=torch.int32, device="cuda").view(4099, 3), q_weight=w)
    first = sa.sparse_attn_norm_rope_backward(g, None, x, **opt)
    for _ in range(3):
        again = sa.sparse_attn_norm_rope_backward(g, None, x, **opt)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sa.sparse_attn_norm_rope(x, **opt)
        made = sa.sparse_attn_norm_rope_backward(g, None, x, **opt)
    x.copy_(make((1, 24, 4099, 128), torch.bfloat16, 5))
    graph.replay()
    torch.cuda.synchronize()
    want = sa.sparse_attn_norm_rope_backward(g, None, x, **opt)
    assert torch.equal(y, sa.sparse_attn_norm_rope(x, **opt))
    assert torch.equal(made[0], want[0]) and torch.equal(made[1], want[1])


def test_offsets_past_32_bits():
    from video_dit_sparse_gb300 import binding as sa
    far = torch.empty(2 ** 31 + 2 ** 27 + 3 * 128, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(far, (2, 1, 3, 128), (2 ** 31 + 2 ** 27, 128, 128, 1))
    x.copy_(make((2, 1, 3, 128), torch.bfloat16, 1))
    opt = dict(axes=(128,), positions=torch.arange(3, dtype=torch.int32, device="cuda")[:, None])
    y = sa.sparse_attn_norm_rope(x, out=torch.empty(2, 1, 3, 128, dtype=torch.bfloat16, device="cuda"), **opt)
    assert torch.equal(y, sa.sparse_attn_norm_rope(x.contiguous(), **opt))
    g = make((2, 1, 3, 128), torch.bfloat16, 2)
    want = sa.sparse_attn_norm_rope_backward(g, None, x.contiguous(), **opt)[0]
    assert torch.equal(sa.sparse_attn_norm_rope_backward(g, None, x, out=torch.empty_like(g), **opt)[0], want)
    sa.sparse_attn_norm_rope(x, out=x, **opt)
    assert torch.equal(x, y)
