"""GPU checks of the rotary positions against the 64-bit form.

Tolerance: the rotation is two products and a sum in fp32 on cosines off by at most 2^-22 (angle 2^-24 of a
half turn, sincospi within two units), so |error| <= 2^-20 (|x| + |y|) of the pair, and one rounding to the output
type (half a step: bf16 2^-8, fp32 2^-24 of the value)."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O

pytestmark = pytest.mark.gpu


def make(shape, dtype, seed, layout="bhnd"):
    g = torch.Generator().manual_seed(seed)
    B, H, N, d = shape
    x = torch.randn((B, H, N, d) if layout == "bhnd" else (B, N, H, d), generator=g).to(dtype).cuda()
    return x if layout == "bhnd" else x.transpose(1, 2)


def check(got, x, pos, axes, half, **kw):
    x64 = x.double().cpu().numpy()
    want = O.rope(x64, pos, axes, half=half, **kw)
    mag = np.abs(x64)
    r = sum(axes)
    pair = np.zeros_like(mag)
    if half:
        pair[..., :r // 2] = pair[..., r // 2:r] = mag[..., :r // 2] + mag[..., r // 2:r]
    else:
        pair[..., 0:r:2] = pair[..., 1:r:2] = mag[..., 0:r:2] + mag[..., 1:r:2]
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -20 * pair
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d,axes", [(128, (44, 42, 42)), (128, (32, 48, 48)), (64, (24, 20, 20)), (64, (16, 8, 8)),
                                    (128, (2, 0, 14))])
@pytest.mark.parametrize("grid,voxel,layout", [((3, 5, 7), None, "bhnd"), ((5, 7, 9), (2, 3, 4), "bnhd"),
                                               ((1, 1, 1), (2, 8, 8), "bhnd")])
def test_grid(dtype, half, d, axes, grid, voxel, layout):
    from video_dit_sparse_gb300 import binding as sa
    N = grid[0] * grid[1] * grid[2]
    q, k = make((2, 5, N, d), dtype, 1, layout), make((2, 2, N, d), dtype, 2, layout)
    off = (1000003, -7, 12)
    y, z = sa.sparse_attn_rope(q, k, axes=axes, grid=grid, voxel=voxel, offset=off,
                               pairing="half" if half else "interleaved")
    pos = O.voxel_positions(grid, voxel, off)
    check(y, q, pos, axes, half)
    check(z, k, pos, axes, half)


@pytest.mark.parametrize("N", [1, 31, 33, 257])
@pytest.mark.parametrize("shared", [True, False])
def test_positions_and_frequencies(N, shared):
    from video_dit_sparse_gb300 import binding as sa
    x = make((3, 4, N, 64), torch.float32, 5)
    rng = np.random.default_rng(N)
    pos = rng.integers(-2 ** 31, 2 ** 31, size=(N, 2) if shared else (3, N, 2))
    # whole-turn fractions that 64-bit products hold exactly at these positions
    freq = [2 * np.pi * j / 4096 for j in range(16)]
    y = sa.sparse_attn_rope(x, axes=(16, 16), inv_freq=freq, pairing="half", inverse=True,
                            positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    turns = np.mod(pos[..., None, :] * np.arange(16)[:, None], 4096)  # per pair and axis, exact
    want = x.double().cpu().numpy().copy()
    for i in range(16):
        t = -2 * np.pi * turns[..., i, 0 if i < 8 else 1] / 4096
        t = t[None, None] if shared else t[:, None]
        a, b = want[..., i].copy(), want[..., i + 16].copy()
        want[..., i], want[..., i + 16] = a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)
    # 2 pi j / 4096 as a double is off by 2^-53 of itself: at 2^31 positions 2^-22 of a radian more
    assert np.abs(y.double().cpu().numpy() - want).max() <= 2.0 ** -18 * 8


def test_gradient_is_the_inverse_and_matches_differences():
    from video_dit_sparse_gb300 import binding as sa
    kw = dict(axes=(24, 20, 20), grid=(2, 3, 5), offset=(9, 0, 0))
    x, g = make((1, 2, 30, 64), torch.float32, 3), make((1, 2, 30, 64), torch.float32, 4)
    gx = sa.sparse_attn_rope(g, inverse=True, **kw)
    # the map is linear: <g, rope(e)> = <gx, e> for every direction e
    for seed in range(4):
        e = make((1, 2, 30, 64), torch.float32, 10 + seed)
        lhs = (g.double() * (sa.sparse_attn_rope(x + e, **kw).double() - sa.sparse_attn_rope(x, **kw).double())).sum()
        rhs = (gx.double() * ((x + e).double() - x.double())).sum()
        # 3840 terms of a few units, each within 2^-20 of them
        assert abs(float(lhs - rhs)) <= 3840 * 2.0 ** -20 * 16
    back = sa.sparse_attn_rope(sa.sparse_attn_rope(x, **kw), inverse=True, **kw)
    assert float((back - x).abs().max()) <= 2.0 ** -19 * 16


def test_in_place_into_a_cache_and_interleaved_views():
    from video_dit_sparse_gb300 import binding as sa
    axes, grid = (44, 42, 42), (2, 4, 5)
    qkv = torch.randn(2, 40, 3, 4, 128, device="cuda").to(torch.bfloat16)
    src = qkv.clone()
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    want_q, want_k = sa.sparse_attn_rope(src[:, :, 0].transpose(1, 2), src[:, :, 1].transpose(1, 2), axes=axes, grid=grid)
    cache = torch.full((2, 4, 200, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    slot = cache[:, :, 80:120]
    sa.sparse_attn_rope(q, k, axes=axes, grid=grid, out=(q, slot))
    assert torch.equal(q, want_q) and torch.equal(slot, want_k)
    assert torch.equal(qkv[:, :, 1:], src[:, :, 1:])
    assert bool((cache[:, :, :80] == 7).all()) and bool((cache[:, :, 120:] == 7).all())


def test_in_place_on_a_fused_projection():
    from video_dit_sparse_gb300 import binding as sa
    qkv = torch.randn(2, 40, 12 + 2 + 2, 64, device="cuda").to(torch.bfloat16)
    src = qkv.clone()
    q, k = (qkv.transpose(1, 2)[:, a:b] for a, b in ((0, 12), (12, 14)))
    want = sa.sparse_attn_rope(src.transpose(1, 2)[:, :14], axes=(24, 20, 20), grid=(2, 4, 5))
    sa.sparse_attn_rope(q, k, axes=(24, 20, 20), grid=(2, 4, 5), out=(q, k))
    assert torch.equal(qkv.transpose(1, 2)[:, :14], want) and torch.equal(qkv[:, :, 14:], src[:, :, 14:])


def test_elements_outside_the_rotation_and_non_finite_rows():
    from video_dit_sparse_gb300 import binding as sa
    for pairing in ("interleaved", "half"):
        x = torch.randn(1, 2, 9, 64, device="cuda")
        x[..., 32:] = float("inf")
        x[0, 1, 3] = float("nan")
        y = sa.sparse_attn_rope(x, axes=(32,), positions=torch.arange(9, device="cuda", dtype=torch.int32)[:, None],
                                pairing=pairing)
        assert bool(torch.isinf(y[0, 0, :, 32:]).all()) and bool(torch.isfinite(y[0, 0, :, :32]).all())
        assert bool(torch.isnan(y[0, 1, 3]).all()) and bool(torch.isfinite(y[0, 1, 4, :32]).all())


def test_stream_graph_and_repeated_input():
    from video_dit_sparse_gb300 import binding as sa
    x = make((2, 3, 50, 128), torch.bfloat16, 8)
    kw = dict(axes=(44, 42, 42), grid=(2, 5, 5))
    want = sa.sparse_attn_rope(x, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sa.sparse_attn_rope(x, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.sparse_attn_rope(x, out=out, **kw)
    x.copy_(make((2, 3, 50, 128), torch.bfloat16, 9))
    g.replay()
    assert torch.equal(out, sa.sparse_attn_rope(x, **kw))
    one = x[:1, :1].expand(2, 3, 50, 128)
    assert torch.equal(sa.sparse_attn_rope(one, **kw)[1, 2], sa.sparse_attn_rope(one[:1, :1], **kw)[0, 0])


@pytest.mark.parametrize("freq", [3.14159, 100.0, 64.7, 1e6, 1.0, 0.8, -2.7182818, 1e-9])
def test_far_positions_of_given_frequencies(freq):
    """The angle p f is reduced exactly, whatever the size of f: a cosine and a sine within 2^-24 half turns of it and
    two units of sincospi."""
    from decimal import Decimal, getcontext
    from video_dit_sparse_gb300 import binding as sa
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -1999999999, 7, 0, 1, -1]
    x = torch.zeros(1, 1, len(pos), 64, device="cuda")
    x[..., 0] = 1.0
    y = sa.sparse_attn_rope(x, axes=(2,), inv_freq=[freq], positions=torch.tensor(pos, dtype=torch.int32, device="cuda")[:, None])
    got = y[0, 0, :, :2].double().cpu().numpy()
    for i, p in enumerate(pos):
        turns = Decimal(freq) * p / (2 * pi)
        t = 2 * np.pi * float(turns - turns.to_integral_value())
        # 2^-24 of a half turn: 2^-24 pi; sincospi: 2^-22; the two products and their sum: 2^-24
        assert np.abs(got[i] - [np.cos(t), np.sin(t)]).max() <= 2.0 ** -24 * np.pi + 2.0 ** -22 + 2.0 ** -24, (p, got[i])
