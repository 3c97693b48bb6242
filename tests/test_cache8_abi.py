"""Refusals of the normalised rotation and of the 8-bit cache (no GPU needed: they come before any CUDA call), and pins of
their 64-bit forms against independent computations."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache8_ops as P
from oracle import cache_ops as O

INVALID, UNSUPPORTED = 1, 2
X, Y, G, W, V, WS, Q, OUT, LSE, K8, V8, KS, VS = (i << 26 for i in range(1, 14))


@pytest.fixture(scope="module")
def sa():
    from video_dit_sparse_gb300 import build
    build.build()
    from video_dit_sparse_gb300 import binding
    return binding


def passes(status):
    """What passes the checks on arguments ends at the device's (on a machine without one)."""
    return torch.cuda.is_available() or status not in (0, INVALID)


# ---------------------------------------------------------------- normalised rotation

def norm(sa, **kw):
    p = sa.sa_norm_rope()
    p.rope = sa.sa_rope(2, 30, 64, 3)
    for i, n in enumerate((24, 20, 20)):
        p.rope.axis_dim[i] = n
    p.rope.theta, p.rope.grid = 1e4, sa.sa_voxel_grid(2, 3, 5, 0, 0, 0)
    p.norm, p.weight_dtype, p.eps = 0, 1, 1e-6
    for n, x in kw.items():
        setattr(p.rope if hasattr(p.rope, n) else p, n, x)
    return p


def strides(sa, H=2):
    return sa.sa_strides(H * 30 * 64, 30 * 64, 64)


def side(sa, **kw):
    s = sa.sa_norm_side(2, X, strides(sa), Y, strides(sa), W, V)
    for n, x in kw.items():
        setattr(s, n, x)
    return s


def grad(sa, **kw):
    s = sa.sa_norm_grad_side(2, X, strides(sa), G, strides(sa), Y, strides(sa), W, V, V + 4096)
    for n, x in kw.items():
        setattr(s, n, x)
    return s


BYTES = 2 * 2 * 30 * 64 * 2  # of a tensor


def test_norm_rope_refusals(sa):
    def call(p, a, b=None):
        return sa.lib.sparse_attn_norm_rope(p, a, b, None)
    ok = norm(sa)
    assert passes(call(ok, side(sa))) and passes(call(ok, side(sa, y=X)))
    assert call(None, side(sa)) == INVALID and call(ok, None) == INVALID
    for bad in (dict(norm=2), dict(weight_dtype=7), dict(eps=-1.0), dict(eps=float("nan")), dict(inverse=1), dict(B=0),
                dict(N=31), dict(theta=0.0), dict(axes=0)):
        assert call(norm(sa, **bad), side(sa)) == INVALID, bad
    for bad in (dict(d=96), dict(B=70000)):
        assert call(norm(sa, **bad), side(sa)) == UNSUPPORTED, bad
    S = sa.sa_strides
    for bad in (dict(H=0), dict(x=None), dict(y=None), dict(x=X + 8), dict(y=Y + 8), dict(y=X + 128), dict(weight=W + 2),
                dict(bias=V + 1), dict(weight=Y + 64), dict(bias=Y), dict(ys=S(3840, 1920, 0)), dict(xs=S(3840, 1920, 60)),
                dict(y=X, ys=S(1920 * 2, 64, 128))):
        assert call(ok, side(sa, **bad)) == INVALID, bad
    # the second side: anywhere but on the first one's tensors
    far = dict(x=X + (1 << 24), y=Y + (1 << 24))
    assert passes(call(ok, side(sa), side(sa, **far)))
    for bad in (dict(x=Y, y=Y + (1 << 24)), dict(x=X + (1 << 24), y=X), dict(x=X + (1 << 24), y=Y),
                dict(x=X + (1 << 24), y=Y + (1 << 24), H=-1)):
        assert call(ok, side(sa), side(sa, **bad)) == INVALID, bad
    assert call(ok, side(sa), side(sa, weight=Y, **far)) == INVALID  # under the first side's output
    assert passes(call(ok, side(sa), side(sa, H=0, x=None, y=None)))


def test_norm_rope_backward_refusals(sa):
    def call(p, a, b=None, ws=WS, n=1 << 24):
        return sa.lib.sparse_attn_norm_rope_backward(p, a, b, ws, n, None)
    ok = norm(sa)
    need = sa.lib.sparse_attn_norm_rope_backward_workspace_size(ok, 2, 0)
    assert need > 0
    assert sa.lib.sparse_attn_norm_rope_backward_workspace_size(norm(sa, norm=3), 2, 0) == 0
    assert sa.lib.sparse_attn_norm_rope_backward_workspace_size(None, 2, 0) == 0
    assert passes(call(ok, grad(sa))) and passes(call(ok, grad(sa, dx=X))) and passes(call(ok, grad(sa, dx=G)))
    assert passes(call(ok, grad(sa, dweight=None, dbias=None), ws=None, n=0))
    assert call(ok, grad(sa), ws=None, n=0) == INVALID and call(ok, grad(sa), n=need - 1) == INVALID
    assert call(ok, grad(sa), ws=WS + 16) == INVALID
    for bad in (dict(x=None), dict(dy=None), dict(dx=None), dict(dx=X + 128), dict(dx=G + 128), dict(dweight=V + 2),
                dict(dbias=V + 4096 + 1), dict(dbias=V), dict(dweight=X), dict(dweight=G + BYTES - 4), dict(dbias=Y),
                dict(dweight=W), dict(weight=Y), dict(dweight=WS)):
        assert call(ok, grad(sa, **bad)) == INVALID, bad
    far = dict(x=X + (1 << 24), dy=G + (1 << 24), dx=Y + (1 << 24), dweight=V + 8192, dbias=None)
    assert passes(call(ok, grad(sa), grad(sa, **far)))
    for bad in (dict(dweight=V), dict(dx=Y), dict(dx=X), dict(dx=G), dict(x=Y), dict(dy=Y)):
        assert call(ok, grad(sa), grad(sa, **{**far, **bad})) == INVALID, bad


# ---------------------------------------------------------------- cache

def cache(sa, **kw):
    c = sa.sa_cache8(2, 3, 100, 128, 32, K8, V8)
    c.ks = c.vs = sa.sa_strides(3 * 100 * 128, 100 * 128, 128)
    c.k_scale, c.v_scale = KS, VS
    c.k_scales = c.v_scales = sa.sa_strides(12, 4, 1)
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def bad_caches(sa, output):
    S = sa.sa_strides
    bad = [dict(B=0), dict(Hkv=0), dict(N=0), dict(d=0), dict(block=0), dict(block=48), dict(block=256), dict(k=None),
           dict(v=None), dict(k=K8 + 8), dict(k_scale=None), dict(v_scale=VS + 2), dict(ks=S(38400, 12800, 120)),
           dict(vs=S(38400, -12800, 128)), dict(k_scales=S(12, -4, 1)), dict(v_scales=S(2 ** 62, 4, 1)),
           dict(ks=S(38400, 0, 128))]
    if output:
        bad += [dict(ks=S(38400, 128, 128)), dict(k_scales=S(12, 3, 1)), dict(v_scales=S(0, 4, 1)), dict(v=K8 + 128),
                dict(v_scale=KS), dict(v_scale=K8), dict(k_scale=V8 + 128)]
    return bad


def test_cache8_append_refusals(sa):
    S = sa.sa_strides
    st = S(3 * 7 * 128, 7 * 128, 128)

    def call(c, n=7, k=X, ks=st, v=Y, vs=st, start=None, at=0, counts=None):
        return sa.lib.sparse_attn_cache8_append(c, n, k, ks, v, vs, start, at, counts, None)
    ok = cache(sa)
    assert passes(call(ok)) and passes(call(ok, ks=S(0, 0, 128)))  # new rows may repeat a dimension
    assert call(None) == INVALID
    for bad in bad_caches(sa, True):
        assert call(cache(sa, **bad)) == INVALID, bad
    for bad in (dict(d=96), dict(N=2 ** 30 + 1), dict(B=2 ** 24)):
        assert call(cache(sa, **bad)) == UNSUPPORTED, bad
    for bad in (dict(n=0), dict(n=-1), dict(k=None), dict(v=None), dict(k=X + 8), dict(ks=None), dict(vs=None),
                dict(start=W + 2), dict(counts=W + 1), dict(k=K8), dict(v=V8 + 1024), dict(k=KS), dict(v=VS - 256)):
        assert call(ok, **bad) == INVALID, bad
    assert call(ok, n=2 ** 30 + 1) == UNSUPPORTED
    # keys and values as halves of one buffer's rows
    both = dict(v=K8 + 128, ks=S(3 * 100 * 256, 100 * 256, 256), vs=S(3 * 100 * 256, 100 * 256, 256))
    assert passes(call(cache(sa, **both)))


def test_cache8_read_refusals(sa):
    S = sa.sa_strides
    st = S(3 * 7 * 128, 7 * 128, 128)

    def call(c, first=None, at=0, n=7, dtype=0, k=X, ks=st, v=Y, vs=st):
        return sa.lib.sparse_attn_cache8_read(c, first, at, n, dtype, k, ks, v, vs, None)
    ok = cache(sa)
    assert passes(call(ok)) and passes(call(ok, k=None, ks=None)) and passes(call(ok, v=None, vs=None))
    assert call(None) == INVALID and call(ok, k=None, v=None) == INVALID
    for bad in bad_caches(sa, False):
        assert call(cache(sa, **bad)) == INVALID, bad
    for bad in (dict(n=0), dict(dtype=3), dict(k=X + 8), dict(ks=None), dict(first=W + 2), dict(v=X + 128), dict(v=X, dtype=1),
                dict(k=K8), dict(v=VS), dict(ks=S(0, 896, 128))):
        assert call(ok, **bad) == INVALID, bad
    assert call(ok, n=2 ** 30 + 1) == UNSUPPORTED


def attend(sa, **kw):
    p = sa.sa_attend8(6, 8, 0.1, 0)
    p.q = p.o = sa.sa_strides(6 * 8 * 128, 8 * 128, 128)
    for n, x in kw.items():
        setattr(p, n, x)
    return p


def test_forward_cache8_refusals(sa):
    size = sa.lib.sparse_attn_forward_cache8_workspace_size

    def call(p, c, q=Q, o=OUT, lse=LSE, status=None, ws=WS, n=1 << 25):
        return sa.lib.sparse_attn_forward_cache8(p, c, q, o, lse, status, ws, n, None)
    ok, c = attend(sa), cache(sa)
    assert passes(call(ok, c)) and passes(call(ok, c, o=Q)) and passes(call(ok, c, lse=None))
    assert call(None, c) == INVALID and call(ok, None) == INVALID and size(None, c) == 0 and size(ok, None) == 0
    for bad in bad_caches(sa, False):
        assert call(ok, cache(sa, **bad)) == INVALID, bad
    for bad in (dict(Hq=0), dict(Hq=5), dict(Nq=0), dict(scale=0.0), dict(scale=float("inf")), dict(scale=3e38), dict(out_dtype=4),
                dict(causal=-1), dict(lengths=W + 1), dict(q=sa.sa_strides(0, 1024, 128)), dict(o=sa.sa_strides(6144, 128, 128))):
        assert call(attend(sa, **bad), c) == INVALID, bad
    for bad in (dict(d=96), dict(N=2 ** 30 + 1)):
        assert call(ok, cache(sa, **bad)) == UNSUPPORTED, bad
    wide = sa.sa_strides(387 * 1024, 1024, 128)
    assert call(attend(sa, Hq=387, q=wide, o=wide), c) == UNSUPPORTED  # 129 heads share one
    for bad in (dict(q=None), dict(o=None), dict(q=Q + 8), dict(o=OUT + 8), dict(lse=LSE + 2), dict(status=W + 1), dict(o=Q + 256),
                dict(o=K8), dict(o=V8 + 256), dict(o=KS - 256), dict(lse=Q), dict(lse=OUT), dict(lse=K8), dict(lse=VS)):
        assert call(ok, c, **bad) == INVALID, bad
    assert call(attend(sa, out_dtype=1), c, o=Q) == INVALID  # fp32 rows are not q's
    long = cache(sa, N=4000, ks=sa.sa_strides(3 * 4000 * 128, 4000 * 128, 128), vs=sa.sa_strides(3 * 4000 * 128, 4000 * 128, 128),
                 k_scales=sa.sa_strides(375, 125, 1), v_scales=sa.sa_strides(375, 125, 1))
    one = attend(sa, Nq=1)
    need = size(one, long)
    assert need > 0 and need % 256 == 0 and size(one, c) == 0  # (short heads are not cut)
    assert call(one, long, ws=None, n=0) == INVALID and call(one, long, n=need - 1) == INVALID
    assert call(one, long, ws=WS + 16) == INVALID and call(one, long, ws=K8) == INVALID and call(one, long, ws=Q) == INVALID
    assert passes(call(one, c, ws=None, n=0))


def test_binding_refusals(sa):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    c = sa.sparse_attn_cache8(1, 2, 16, 64, block=16, device="cpu")
    assert c.k.dtype is torch.float8_e4m3fn and c.k_scale.shape == (1, 2, 1) and c.block == 16
    for f in (lambda: sa.sparse_attn_norm_rope(x, axes=(64,), grid=(1, 2, 2)),
              lambda: sa.sparse_attn_norm_rope(x, norm="batch", axes=(64,), grid=(1, 2, 2)),
              lambda: sa.sparse_attn_norm_rope(x.half(), axes=(64,), grid=(1, 2, 2)),
              lambda: sa.sparse_attn_norm_rope_backward(x, None, x, x, axes=(64,), grid=(1, 2, 2)),
              lambda: sa.sparse_attn_cache8_append(c, x, x, 0),
              lambda: sa.sparse_attn_cache8_read(c, 0, 4),
              lambda: sa.sparse_attn_forward_cache8(x, c)):
        with pytest.raises(ValueError):
            f()


def test_binding_takes_no_position_that_does_not_fit(sa):
    """A number that a 32-bit argument would wrap around must not end up at another token."""
    assert sa._tokens(5, "start", 0, 1) == (0, 5) and sa._tokens(-2 ** 31, "start", 0, 1) == (0, -2 ** 31)
    for at in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            sa._tokens(at, "start", 0, 1)
    for block in (0, 8, 48, 256):
        with pytest.raises(ValueError):
            sa.sparse_attn_cache8(1, 1, 16, 64, block=block, device="cpu")


# ---------------------------------------------------------------- pins of the 64-bit forms

def test_norm_form_against_torch():
    rng = np.random.default_rng(0)
    x, w, b, dy = rng.normal(size=(2, 3, 5, 16)), rng.normal(size=16), rng.normal(size=16), rng.normal(size=(2, 3, 5, 16))
    pos = rng.integers(-9, 9, size=(5, 2))
    t = [torch.from_numpy(v).requires_grad_() for v in (x, w, b)]
    for layer in (False, True):
        for half in (False, True):
            if layer:
                y = torch.nn.functional.layer_norm(t[0], (16,), t[1], t[2], eps=1e-3)
            else:
                y = torch.nn.functional.rms_norm(t[0], (16,), t[1], eps=1e-3) + t[2]
            cols = [O.rope(np.broadcast_to(np.eye(16)[i], (1, 1, 5, 16)), pos, (8, 8), half=half)[0, 0] for i in range(16)]
            turn = torch.from_numpy(np.stack(cols, 1))  # [N, from, to]
            y = torch.einsum("bhni,nio->bhno", y, turn)
            assert np.allclose(y.detach().numpy(), P.norm_rope(x, pos, (8, 8), layer, 1e-3, w, b, half=half))
            got = torch.autograd.grad(y, t, torch.from_numpy(dy))
            for g, want in zip(got, P.norm_rope_grad(dy, x, pos, (8, 8), layer, 1e-3, w, half=half)):
                assert np.allclose(g.numpy(), want)


def test_codes_against_torch():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)).mul(60).clamp(-448, 448)
    x = torch.cat([x, x * 2.0 ** -12, torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 17.0, 19.0])])
    assert np.array_equal(P.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    every = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(P.decode(every.numpy()), every.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    assert np.isnan(P.decode(P.encode([np.inf, -np.inf, np.nan]))).all()


def test_append_form():
    rng = np.random.default_rng(2)
    codes, scales = np.zeros((40, 4), np.uint8), np.zeros(3)
    x = rng.normal(size=(20, 4))
    codes, scales = P.append(codes, scales, x, 0, 20, 16)
    assert (np.abs(P.values(codes, scales, 16)[:20] - x) <= np.abs(x) * 2.0 ** -4 + np.repeat(scales, 16)[:20, None] * 2.0 ** -10).all()
    assert scales[2] == 0 and scales[0] <= np.abs(x).max() / 224  # (448 / 2 is reached: the least power of two)
    grown, s2 = P.append(codes, scales, 8 * x[:1], 20, 1, 16)
    assert s2[1] > scales[1] and s2[0] == scales[0] and np.array_equal(grown[:16], codes[:16])
    old, new = P.values(codes, scales, 16)[16:20], P.values(grown, s2, 16)[16:20]
    assert (np.abs(new - old) <= s2[1] * 2.0 ** -10).all()  # by whole binades: only the smallest are rounded again
    less, s3 = P.append(grown, s2, x[:1] * 1e-3, 21, 1, 16)
    assert s3[1] == s2[1] and np.array_equal(less[:21], grown[:21])
    assert P.append(codes, scales, x, 50, 20, 16)[0] is not codes and np.array_equal(P.append(codes, scales, x, 50, 20, 16)[0], codes)
    assert P.held(float("inf")) == P.held(-1.0) == P.held(float("nan")) == 0.0 and P.held(2.0) == 2.0


def test_row_ends_are_those_of_the_masked_attention():
    for Nq, n, causal in ((3, 9, 1), (5, 9, 3), (4, 2, 1), (7, 7, 0), (2, 0, 1), (6, 10, 4)):
        see, _ = O.visible(Nq, max(n, 1), causal, length=n)
        assert P.row_ends(Nq, n, causal).tolist() == see.sum(1).tolist()
