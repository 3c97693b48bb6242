"""Refusals of the operators around the attention path (no GPU needed: they come before any CUDA call), and pins of
their 64-bit forms against independent computations."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as O

INVALID, UNSUPPORTED = 1, 2
A16, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def sa():
    from video_dit_sparse_gb300 import build
    build.build()
    from video_dit_sparse_gb300 import binding
    return binding


def masked(sa, **kw):
    p = sa.sa_masked(1, 4, 2, 8, 64, 128, 0.1, 0)
    p.q = sa.sa_strides(4 * 8 * 128, 8 * 128, 128)
    p.k = sa.sa_strides(2 * 64 * 128, 64 * 128, 128)
    p.v, p.o = p.k, p.q
    for n, x in kw.items():
        setattr(p, n, x)
    return p


Q, K, V, OUT, WS, LSE = (i << 24 for i in range(1, 7))


def forward(sa, p, q=Q, k=K, v=V, o=OUT, lse=None, ws=WS, nws=1 << 30):
    return sa.lib.sparse_attn_forward_masked(p, q, k, v, o, lse, None, ws, nws, None)


def test_forward_masked_refusals(sa):
    assert forward(sa, None) == INVALID
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Nq=0), dict(Nk=0), dict(d=0), dict(Hq=3), dict(scale=0.0),
                dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf")), dict(causal=-1), dict(ndocs=-1),
                dict(out_dtype=5), dict(scale=3e38), dict(cap=1e-38, scale=1e5), dict(ndocs=2),
                dict(ndocs=2, docs_q=A16), dict(docs_q=A16), dict(prefix=A16),
                dict(ndocs=1, docs_q=A16, docs_k=A16, lengths=A16), dict(slopes=A16 + 2), dict(lengths=A16 + 1)):
        assert forward(sa, masked(sa, **bad)) == INVALID, bad
    for bad in (dict(d=96), dict(Nk=2 ** 30 + 1), dict(Nq=2 ** 30 + 1), dict(B=2 ** 23)):
        assert forward(sa, masked(sa, **bad)) == UNSUPPORTED, bad
    ok = masked(sa)
    for name in ("q", "k", "v", "o"):
        assert forward(sa, ok, **{name: None}) == INVALID
        assert forward(sa, ok, **{name: MIS}) == INVALID
    wide = sa.sa_strides(258 * 1024, 1024, 128)
    assert forward(sa, masked(sa, Hq=258, q=wide, o=wide)) == UNSUPPORTED
    assert forward(sa, ok, lse=LSE + 2) == INVALID
    if not torch.cuda.is_available():  # what passes the checks on arguments ends at the device's
        assert forward(sa, ok) not in (0, INVALID) and forward(sa, ok, o=Q) not in (0, INVALID)
    for bad in (dict(o=K), dict(o=V + 256), dict(o=Q + 256), dict(lse=K), dict(lse=OUT), dict(lse=Q + 64)):
        assert forward(sa, ok, **bad) == INVALID, bad
    assert forward(sa, masked(sa, out_dtype=1), o=Q) == INVALID  # fp32 rows are not q's
    S = sa.sa_strides
    for bad in (dict(q=S(4096, 1024, -128)), dict(q=S(4096, 1024, 100)), dict(k=S(16384, 8192, 0)),
                dict(o=S(4096, 1024, 0)), dict(o=S(4096, 128, 128)), dict(o=S(4096, 1024, 64)),
                dict(v=S(16384, 2 ** 40, 128))):
        assert forward(sa, masked(sa, **bad)) == INVALID, bad
    need = sa.lib.sparse_attn_forward_masked_workspace_size(ok)
    assert need == 0  # one tile of keys: nothing to split
    few = masked(sa, Nq=1, Nk=28160, q=S(512, 128, 128), o=S(512, 128, 128), k=S(0, 28160 * 128, 128),
                 v=S(0, 28160 * 128, 128))
    need = sa.lib.sparse_attn_forward_masked_workspace_size(few)
    assert need > 0 and need % 256 == 0
    assert forward(sa, few, ws=None, nws=0) == INVALID
    assert forward(sa, few, nws=need - 1) == INVALID
    assert forward(sa, few, ws=WS + 16) == INVALID and forward(sa, few, ws=K) == INVALID
    assert sa.lib.sparse_attn_forward_masked_workspace_size(None) == 0
    for big in (dict(Hq=2 ** 24, Hkv=2 ** 24, Nq=2 ** 30), dict(Hq=2 ** 22, Hkv=2 ** 22, Nq=2 ** 18 + 1),
                dict(Hq=128, Hkv=1, Nq=2 ** 30, B=2)):  # products of these do not fit 32 bits
        assert sa.lib.sparse_attn_forward_masked_workspace_size(masked(sa, Nk=1, **big)) == 0, big
    assert sa.lib.sparse_attn_forward_masked_workspace_size(masked(sa, d=96)) == 0


def test_cache_weights_refusals(sa):
    W = 0x4000000

    def call(p, q=A16, k=A16, lse=A16, w=W, o=W, decay=1.0):
        return sa.lib.sparse_attn_cache_weights(p, q, k, lse, w, o, decay, None, None)
    ok = masked(sa)
    assert call(None) == INVALID
    for bad in (dict(q=None), dict(k=None), dict(lse=None), dict(o=None), dict(w=None), dict(q=MIS), dict(lse=A16 + 1),
                dict(w=W + 2), dict(o=W + 2), dict(decay=float("nan")), dict(o=W + 256), dict(lse=W + 4),
                dict(q=W), dict(k=W)):
        assert call(ok, **bad) == INVALID, bad
    assert call(masked(sa, q=sa.sa_strides(0, 0, 128))) == INVALID  # a repeated head
    assert call(masked(sa, Hq=600, Hkv=2, q=sa.sa_strides(600 * 1024, 1024, 128))) == UNSUPPORTED


def test_cache_evict_refusals(sa):
    S = sa.sa_strides
    at = {n: (i + 1) << 24 for i, n in enumerate(("w", "k", "v", "kept", "ko", "vo", "wo"))}

    def prob(**kw):
        p = sa.sa_evict(1, 2, 64, 128, 16, 4, 4)
        p.k = p.v = S(64 * 256, 64 * 128, 128)
        p.k_out = p.v_out = S(16 * 256, 16 * 128, 128)
        for n, x in kw.items():
            setattr(p, n, x)
        return p

    def call(p, **kw):
        t = dict(at, **kw)
        return sa.lib.sparse_attn_cache_evict(p, t["w"], t["k"], t["v"], t["kept"], t["ko"], t["vo"], t["wo"], None)
    assert call(None) == INVALID
    for bad in (dict(B=0), dict(Hkv=0), dict(Nk=0), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=13),
                dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(lengths=A16 + 2), dict(k=S(1, 1, 1)),
                dict(k_out=S(16 * 256, 16 * 128, 64)), dict(v_out=S(0, 0, 128))):
        assert call(prob(**bad)) == INVALID, bad
    for bad in (dict(d=96), dict(B=65536, Hkv=1), dict(Nk=2 ** 30 + 1), dict(budget=2 ** 30 + 1)):
        assert call(prob(**bad)) == UNSUPPORTED, bad
    ok = prob()
    for bad in (dict(w=None), dict(kept=None), dict(k=None), dict(vo=None), dict(ko=at["k"]), dict(vo=at["v"] + 4096),
                dict(wo=at["w"]), dict(kept=at["w"]), dict(ko=at["vo"]), dict(kept=at["wo"]), dict(k=at["k"] + 8)):
        assert call(ok, **bad) == INVALID, bad


def test_rope_refusals(sa):
    S = sa.sa_strides
    st = S(2 * 30 * 64, 30 * 64, 64)
    X, Y = 1 << 24, 2 << 24

    def prob(**kw):
        p = sa.sa_rope(1, 30, 64, 3)
        for i, n in enumerate(kw.pop("dims", (24, 20, 20))):
            p.axis_dim[i] = n
        p.theta = 1e4
        p.grid = sa.sa_voxel_grid(2, 3, 5, 0, 0, 0)
        for n, x in kw.items():
            setattr(p, n, x)
        return p

    def call(p, H=2, x=X, xs=st, y=Y, ys=st, H1=0, x1=None, x1s=None, y1=None, y1s=None):
        return sa.lib.sparse_attn_rope(p, H, x, xs, y, ys, H1, x1, x1s, y1, y1s, None)
    assert call(None) == INVALID
    nan = (ctypes.c_double * 32)(*([float("nan")] * 32))
    for bad in (dict(B=0), dict(N=0), dict(d=0), dict(axes=0), dict(axes=4), dict(pairing=2), dict(dtype=9),
                dict(theta=0.0), dict(theta=float("inf")), dict(dims=(3, 20, 20)), dict(dims=(-2, 20, 20)), dict(dims=(24, 24, 24)),
                dict(dims=(0, 0, 0)), dict(N=31), dict(axes=2), dict(voxel_order=1), dict(positions=A16 + 2),
                dict(positions=A16, positions_b=-1), dict(positions=A16, positions_b=89), dict(inv_freq=nan),
                dict(grid=sa.sa_voxel_grid(30, 2 ** 31 - 1, 1, 0, 0, 0))):
        assert call(prob(**bad)) == INVALID, bad
    far = prob()
    far.offset[1] = 2 ** 31 - 2
    assert call(far) == INVALID
    for bad in (dict(d=96), dict(pairing=1, dims=(10, 10, 10)), dict(B=70000)):
        assert call(prob(**bad)) == UNSUPPORTED, bad
    # two slots of one buffer interleave; a row less apart they would meet
    two = prob(N=2, grid=sa.sa_voxel_grid(1, 1, 2, 0, 0, 0))
    wide = S(0, 64, 3 * 2 * 64)
    if not torch.cuda.is_available():
        assert call(two, xs=wide, ys=wide, y=X + 2 * 2 * 64) != INVALID
    assert call(two, xs=wide, ys=wide, y=X + 2 * 64) == INVALID
    ok = prob()
    for bad in (dict(H=0), dict(H1=-1), dict(x=None), dict(y=None), dict(xs=None), dict(ys=None), dict(x=X + 8),
                dict(H1=2), dict(H1=2, x1=X, x1s=st, y1=None, y1s=st), dict(y=X + 3840), dict(ys=S(1920, 960, 64)),
                dict(y=X, ys=S(3840, 64, 128))):
        assert call(ok, **bad) == INVALID, bad


def test_views_of_one_buffer(sa):
    """Heads of a fused projection [B, N, Hq + 2 Hkv, d]: views that interleave pass the checks, views that meet do not."""
    Hq, Hk, N, d = 12, 2, 40, 128
    st = sa.sa_strides(N * (Hq + 2 * Hk) * d, d, (Hq + 2 * Hk) * d)
    q, k, v = Q, Q + Hq * d * 2, Q + (Hq + Hk) * d * 2
    p = masked(sa, B=2, Hq=Hq, Hkv=Hk, Nq=N, Nk=N, q=st, k=st, v=st, o=st)
    rope = sa.sa_rope(2, N, d, 3)
    rope.axis_dim[0], rope.theta, rope.grid = 64, 1e4, sa.sa_voxel_grid(1, 5, 8, 0, 0, 0)

    def turn(x1, y1, H1=Hk, x0=q, y0=q):
        return sa.lib.sparse_attn_rope(rope, Hq, x0, st, y0, st, H1, x1, st, y1, st, None)
    if not torch.cuda.is_available():
        assert forward(sa, p, q, k, v, o=q) not in (0, INVALID)
        assert turn(k, k) not in (0, INVALID) and turn(v, k) not in (0, INVALID)
        assert turn(k, k, H1=1) not in (0, INVALID)
    row = d * 2
    for o in (k, v, q + row, q - row, k - row, v + row):
        assert forward(sa, p, q, k, v, o=o) == INVALID
    for x1, y1 in ((k, q), (q, k), (k - row, k - row), (v + row, v + row), (q, q)):
        assert turn(x1, y1) == INVALID
    assert turn(v, v, H1=3) == INVALID  # three heads from v's reach the next token's q


def test_binding_refusals(sa):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    for f in (lambda: sa.sparse_attn_rope(x, axes=(64,), positions=torch.zeros(4, 1, dtype=torch.int32)),
              lambda: sa.sparse_attn_rope(x.half(), axes=(64,), grid=(1, 2, 2)),
              lambda: sa.sparse_attn_forward_masked(x, x, x),
              lambda: sa.sparse_attn_cache_weights(x, x, torch.zeros(1, 2, 4)),
              lambda: sa.sparse_attn_cache_evict(torch.zeros(1, 2, 4), None, None, 2)):
        with pytest.raises(ValueError):
            f()


# ---------------------------------------------------------------- pins of the 64-bit forms

def test_rope_form_is_a_rotation_by_relative_position():
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 1, 1, 6, 32))
    for half in (False, True):
        for axes in ((32,), (8, 16, 8)):
            pos = rng.integers(-50, 50, size=(6, len(axes)))
            a, b = O.rope(x, pos, axes, half=half), O.rope(y, pos, axes, half=half)
            assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1))
            c, e = O.rope(x, pos + 1000, axes, half=half), O.rope(y, pos + 1000, axes, half=half)
            assert np.allclose((a * b).sum(-1), (c * e).sum(-1))
            # products between tokens depend on the difference of their positions alone
            assert np.allclose(a[0, 0] @ b[0, 0].T, c[0, 0] @ e[0, 0].T)
            assert np.allclose(O.rope(a, pos, axes, half=half, inverse=True), x)
    one = np.zeros((1, 1, 1, 4))
    one[..., 0] = 1
    assert np.allclose(O.rope(one, [[3]], (4,)), [np.cos(3), np.sin(3), 0, 0])
    assert np.allclose(O.rope(one, [[3]], (4,), half=True), [np.cos(3), 0, np.sin(3), 0])
    one = one[..., ::-1]
    assert np.allclose(O.rope(one, [[3]], (4,)), [0, 0, -np.sin(0.03), np.cos(0.03)])


def test_attention_form_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 16)), rng.normal(size=(9, 16)), rng.normal(size=(9, 16))
    see, dist = O.visible(5, 9, causal=1)
    assert see.sum() == 5 + 6 + 7 + 8 + 9 and dist[0, 0] == 4 and dist[4, 8] == 0
    t = [torch.from_numpy(x)[None] for x in (q, k, v)]
    want = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=torch.from_numpy(see), scale=0.3)
    o, lse, _ = O.attention(q, k, v, 0.3, see)
    assert np.allclose(o, want[0].numpy())
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(np.where(see, 0.3 * q @ k.T, -np.inf)), -1).numpy())
    p = sum(O.cache_weights(q[i:i + 1], k, lse[i:i + 1], 0.3, see[i:i + 1]) for i in range(5))
    assert np.allclose(p.sum(), 5) and np.allclose(p @ v, o.sum(0))
    # a frame of 3: rows at positions 4..8 of 9
    see, _ = O.visible(5, 9, causal=3)
    assert [int(r.sum()) for r in see] == [6, 6, 9, 9, 9]
    see, _ = O.visible(3, 9, causal=1, docs_q=[0, 1, 3], docs_k=[0, 4, 9], prefix=[0, 2])
    assert see.tolist() == [[j < 4 for j in range(9)], [4 <= j < 8 for j in range(9)], [j >= 4 for j in range(9)]]
    assert not O.visible(3, 2, causal=1)[0][0].any()  # more rows than keys: the first see nothing


def test_evict_form():
    assert O.evict([5, 1, 4, 4, 2, 4], 6, 3, 0, 0).tolist() == [0, 2, 3]
    assert O.evict([0, 1, 4, 4, 2, 0], 6, 4, 1, 1).tolist() == [0, 2, 3, 5]
    assert O.evict([0, np.nan, -np.inf, 0], 4, 3, 0, 0).tolist() == [0, 2, 3]
    assert O.evict([0.0, -0.0, 0.0], 3, 2, 0, 0).tolist() == [0, 1]
    assert O.evict([3, 2, 1], 2, 2, 0, 0).tolist() == [0, 1]


def test_rope_refuses_positions_beyond_any_memory(sa):
    """A stride whose bytes do not fit 64 bits must not pass as a short one."""
    p = sa.sa_rope(3, 30, 64, 1)
    p.axis_dim[0], p.theta, p.positions = 64, 1e4, A16
    st = sa.sa_strides(2 * 30 * 64, 30 * 64, 64)
    for far in (2 ** 61, 2 ** 62, 2 ** 63 - 1, 2 ** 41):
        p.positions_b = far
        assert sa.lib.sparse_attn_rope(p, 2, 1 << 24, st, 2 << 24, st, 0, None, None, None, None, None) == INVALID


def test_more_documents_than_their_indexes_hold_are_refused(sa):
    """Indexes of documents, and sums of two of them, are 32-bit."""
    for n in (2 ** 30 + 1, 2 ** 31 - 1):
        p = masked(sa, B=2, ndocs=n, docs_q=A16, docs_k=A16)
        assert forward(sa, p) == UNSUPPORTED
        assert sa.lib.sparse_attn_cache_weights(p, Q, K, LSE, None, OUT, 0.0, None, None) == UNSUPPORTED
