"""GPU checks of the masked forward against the 64-bit form.

Tolerances.  A score is off by at most e = d 2^-23 a (a: the largest scale * sum |q k| of the row's head, fp32
accumulation of exact products) + 2^-20 cap + 2^-22 bias terms; P is rounded to bf16 (half a step, 2^-8) and O is
normalised by the rounded sum, so
    |o - want| <= (2^-8 + 2 e + 2^-16) 1.01 (sum p |v| + |want|) + the output's own rounding,
    |lse - want| <= e + 2^-20 (1 + |want|)."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O

pytestmark = pytest.mark.gpu


def tensors(B, H, Hk, Nq, Nk, d, seed=0, layout="bhnd", sigma=1.5):
    g = torch.Generator().manual_seed(seed)

    def t(h, n, s):
        x = torch.randn((B, h, n, d) if layout == "bhnd" else (B, n, h, d), generator=g).mul(s).to(torch.bfloat16).cuda()
        return x if layout == "bhnd" else x.transpose(1, 2)
    return t(H, Nq, sigma), t(Hk, Nk, 1.0), t(Hk, Nk, 1.0)


def check(o, lse, q, k, v, *, scale=None, cap=0.0, slopes=None, causal=0, docs_q=None, docs_k=None, prefix=None,
          lengths=None):
    B, H, Nq, d = q.shape
    Hk, Nk = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    eps = torch.finfo(o.dtype).eps / 2
    got, glse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    row = lambda t, b: None if t is None else np.atleast_2d(t)[b % np.atleast_2d(t).shape[0]]  # noqa: E731
    for b in range(B):
        see, dist = O.visible(Nq, Nk, causal, row(docs_q, b), row(docs_k, b), row(prefix, b),
                              None if lengths is None else lengths[b])
        for h in range(H):
            hk = h // (H // Hk)
            sl = 0.0 if slopes is None else float(slopes[h])
            want, wlse, pv = O.attention(q[b, h], k[b, hk], v[b, hk], scale, see, cap=cap, slope=sl, dist=dist)
            kk = np.where(see.any(0)[:, None], k[b, hk], 0.0)
            a = abs(scale) * float((np.abs(q[b, h]) @ np.abs(kk).T).max(initial=0.0))
            e = d * 2.0 ** -23 * a + 2.0 ** -20 * cap + 2.0 ** -22 * abs(sl) * float(dist.max(initial=0.0))
            tol = (2.0 ** -8 + 2 * e + 2.0 ** -16) * 1.01 * (pv + np.abs(want)) + eps * np.abs(want)
            err = np.abs(got[b, h] - want)
            assert (err <= tol).all(), (b, h, float((err - tol).max()), np.argwhere(~(err <= tol))[:4])
            none = np.isinf(wlse)
            assert np.array_equal(glse[b, h] == -np.inf, none)
            assert (got[b, h][none] == 0).all()
            lerr = np.abs(glse[b, h][~none] - wlse[~none])
            assert (lerr <= (e + 2.0 ** -20 * (1 + np.abs(wlse[~none])))).all(), float(lerr.max())


def run(q, k, v, **kw):
    from video_dit_sparse_gb300 import binding as sa
    dev = dict(kw)
    for n in ("docs_q", "docs_k", "prefix", "lengths"):
        if dev.get(n) is not None:
            dev[n] = torch.tensor(dev[n], dtype=torch.int32, device="cuda")
    if dev.get("slopes") is not None:
        dev["slopes"] = torch.tensor(dev["slopes"], dtype=torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sa.sparse_attn_forward_masked(q, k, v, status=status, **dev)
    assert int(status) == 0
    return o, lse


# rows per key head under, at and over one tile; one key to several tiles; odd sizes
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,Nk", [(1, 1, 1, 1), (2, 2, 1, 129), (2, 1, 130, 128), (3, 1, 43, 257), (8, 1, 17, 640),
                                        (2, 2, 300, 77), (6, 2, 100, 513), (1, 1, 515, 1000)])
@pytest.mark.parametrize("causal", [0, 1, 97])
def test_sizes(d, H, Hk, Nq, Nk, causal):
    q, k, v = tensors(2, H, Hk, Nq, Nk, d, seed=Nq + Nk)
    check(*run(q, k, v, causal=causal), q, k, v, causal=causal)


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("H,Hk,Nq,Nk", [(4, 2, 1, 700), (4, 2, 200, 333), (2, 2, 257, 257)])
def test_cap_and_bias(layout, cap, bias, H, Hk, Nq, Nk):
    q, k, v = tensors(2, H, Hk, Nq, Nk, 128, seed=3, layout=layout, sigma=4.0)
    kw = dict(cap=cap, slopes=[2.0 ** -i for i in range(1, H + 1)] if bias else None, causal=1)
    check(*run(q, k, v, out_dtype=torch.float32, **kw), q, k, v, **kw)


DOCS = [
    ([0, 100, 100, 101, 300], [0, 250, 260, 260, 400]),
    ([5, 100, 290], [10, 10, 390]),      # rows and keys of no document, a document without keys
    ([0, 0, 0, 300], [0, 7, 130, 400]),  # documents without rows
    ([0, 300], [0, 0]),                  # nothing to see
]


@pytest.mark.parametrize("dq,dk", DOCS)
@pytest.mark.parametrize("causal,prefix", [(0, None), (1, None), (1, 30), (97, 200)])
def test_documents(dq, dk, causal, prefix):
    q, k, v = tensors(1, 3, 1, 300, 400, 64, seed=7)
    px = None if prefix is None else [prefix] * (len(dq) - 1)
    kw = dict(docs_q=dq, docs_k=dk, prefix=px, causal=causal)
    check(*run(q, k, v, **kw), q, k, v, **kw)


def test_documents_of_each_batch_entry():
    q, k, v = tensors(2, 2, 2, 90, 160, 128, seed=8)
    kw = dict(docs_q=[[0, 30, 90], [0, 89, 90]], docs_k=[[0, 150, 160], [0, 1, 2]], prefix=[[3, 0], [1, 1]], causal=1)
    check(*run(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("Nq", [1, 3, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_lengths_and_what_lies_behind_them(Nq, bad):
    lengths = [0, 1, 127, 128, 300, 400]
    q, k, v = tensors(6, 4, 2, Nq, 400, 128, seed=9)
    for b, n in enumerate(lengths):
        k[b, :, n:] = bad
        v[b, :, n:] = bad
    kw = dict(lengths=lengths, causal=1)
    check(*run(q, k, v, **kw), q, k, v, **kw)
    check(*run(q, k, v, lengths=lengths), q, k, v, lengths=lengths)


def test_non_finite_rows_of_another_document_do_not_leak():
    q, k, v = tensors(1, 1, 1, 256, 512, 64, seed=10)
    kw = dict(docs_q=[0, 128, 256], docs_k=[0, 100, 512])
    o, lse = run(q, k, v, **kw)
    v[0, 0, 100:] = float("nan")
    k[0, 0, 100:] = float("nan")
    q[0, 0, 128:] = float("nan")
    o2, lse2 = run(q[:, :, :128], k, v, docs_q=[0, 128], docs_k=[0, 100])
    assert torch.equal(o2, o[:, :, :128]) or float((o2 - o[:, :, :128]).abs().max()) < 2.0 ** -7 * 4
    assert bool(torch.isfinite(o2).all())


def test_late_maximum_raises_the_reference():
    q, k, v = tensors(1, 2, 2, 200, 640, 128, seed=11)
    k[:, :, 500:] *= 12  # scores far above those of the first tiles
    check(*run(q, k, v, out_dtype=torch.float32), q, k, v)
    k[:, :, :130] *= 12
    check(*run(q, k, v, causal=1, out_dtype=torch.float32), q, k, v, causal=1)


def test_negative_scale_and_far_bias():
    q, k, v = tensors(1, 2, 2, 140, 300, 64, seed=12)
    check(*run(q, k, v, scale=-0.2), q, k, v, scale=-0.2)
    kw = dict(slopes=[50.0, -0.05], causal=0)  # nearly one-hot rows; a bias that grows with distance
    check(*run(q, k, v, **kw), q, k, v, **kw)


def test_strided_views_and_out():
    from video_dit_sparse_gb300 import binding as sa
    buf = torch.randn(2, 70, 3, 4, 64, device="cuda").to(torch.bfloat16)
    q, k, v = (buf[:, :, i].transpose(1, 2) for i in range(3))
    out = torch.full((2, 70, 6, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :, 1:5].transpose(1, 2)
    o, lse = sa.sparse_attn_forward_masked(q, k, v, causal=1, out=view)
    check(o, lse, q, k, v, causal=1)
    assert bool((out[:, :, 0] == 9).all()) and bool((out[:, :, 5] == 9).all())
    cache = torch.randn(2, 4, 500, 64, device="cuda").to(torch.bfloat16)
    kc, vc = cache[:, :, 20:90], cache[:, :, 200:270]
    check(*sa.sparse_attn_forward_masked(q, kc, vc), q, kc, vc)


def test_matches_the_dense_forward():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(1, 2, 2, 384, 1000, 128, seed=13)
    o, lse = sa.sparse_attn_forward_masked(q, k, v, out_dtype=torch.float32)
    d, dl = sa.sparse_attn_forward(q, k, v, None, None, out_dtype=torch.float32)
    assert float((o - d).abs().max()) <= 2.0 ** -7 * 4  # two roundings of P, values within 4 or so
    assert float((lse - dl).abs().max()) <= 2.0 ** -18 * 16


def test_streams_graphs_and_repeatability():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(2, 4, 2, 1, 3000, 128, seed=14)
    kw = dict(causal=1, lengths=torch.tensor([2999, 1234], dtype=torch.int32, device="cuda"))
    want, wl = sa.sparse_attn_forward_masked(q, k, v, **kw)
    for _ in range(3):
        o, l = sa.sparse_attn_forward_masked(q, k, v, **kw)
        assert torch.equal(o, want) and torch.equal(l, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, l = sa.sparse_attn_forward_masked(q, k, v, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.sparse_attn_forward_masked(q, k, v, out=out, lse=lse, **kw)
    kw["lengths"].copy_(torch.tensor([5, 3000], dtype=torch.int32))  # a replay reads the tables anew
    g.replay()
    want, wl = sa.sparse_attn_forward_masked(q, k, v, **kw)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_tables_that_point_outside_read_nothing_outside():
    q, k, v = tensors(1, 2, 2, 150, 200, 64, seed=15)
    big = 2 ** 31 - 1
    for dq, dk in (([0, 150], [-5, 10 ** 6]), ([-10 ** 9, 10 ** 9], [-10 ** 9, 10 ** 9]), ([90, 10, 150], [150, 3, 77]),
                   ([0, 70, 150], [big, -big, big])):
        for causal in (0, 1, big):
            o, lse = run(q, k, v, docs_q=dq, docs_k=dk, causal=causal, prefix=[big] * (len(dq) - 1))
            assert bool(torch.isfinite(o).all())
    o, lse = run(q, k, v, lengths=[10 ** 9])
    check(o, lse, q, k, v)
    o, lse = run(q, k, v, lengths=[-4])
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("d,R,causal,bias", [(64, 1, 1, True), (128, 3, 0, False), (128, 1, 50, False)])
def test_more_units_than_blocks(d, R, causal, bias):
    """Every block takes several units, of different lengths, and the last ones are split."""
    H = 42 * R
    q, k, v = tensors(2, H, 42, 515 // R, 500, d, seed=21)
    kw = dict(causal=causal, slopes=[0.02 * (h % 5) for h in range(H)] if bias else None,
              docs_q=[[0, 60, 61, 515 // R], [0, 0, 100, 515 // R]], docs_k=[[0, 100, 130, 500], [0, 250, 257, 499]])
    check(*run(q, k, v, **kw), q, k, v, **kw)


def test_most_heads_that_share_a_key_head():
    q, k, v = tensors(1, 128, 1, 3, 300, 64, seed=22)
    check(*run(q, k, v, causal=1), q, k, v, causal=1)


def test_offsets_past_32_bits():
    from video_dit_sparse_gb300 import binding as sa
    n, d, far = 300, 64, 1 << 31  # heads 2^31 elements apart
    buf = torch.empty(far + 4 * n * d, dtype=torch.bfloat16, device="cuda")
    views = [buf.as_strided((1, 2, n, d), (0, far, d, 1), i * n * d) for i in range(4)]
    q, k, v = tensors(1, 2, 2, n, n, d, seed=23)
    for to, of in zip(views, (q, k, v)):
        to.copy_(of)
    o, lse = sa.sparse_attn_forward_masked(*views[:3], causal=1, out=views[3])
    want, wl = sa.sparse_attn_forward_masked(q, k, v, causal=1)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    w = sa.sparse_attn_cache_weights(views[0], views[1], lse, causal=1)
    assert torch.equal(w, sa.sparse_attn_cache_weights(q, k, lse, causal=1))
    kept, k2, v2, w2 = sa.sparse_attn_cache_evict(w, views[1], views[2], 100)
    at = kept.long()[..., None].expand(1, 2, 100, d)
    assert torch.equal(k2, k.gather(2, at)) and torch.equal(v2, v.gather(2, at))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    got = sa.sparse_attn_rope(views[0], views[1], axes=(d,), positions=pos, out=(views[3], views[1]))
    assert torch.equal(got[0], sa.sparse_attn_rope(q, axes=(d,), positions=pos))
    assert torch.equal(got[1], sa.sparse_attn_rope(k, axes=(d,), positions=pos))


def test_two_streams_at_once():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(1, 4, 4, 700, 900, 128, seed=24)
    t, kc, vc = tensors(2, 8, 2, 1, 5000, 128, seed=25)
    a = sa.sparse_attn_forward_masked(q, k, v, causal=1)
    b = sa.sparse_attn_forward_masked(t, kc, vc)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        x = sa.sparse_attn_forward_masked(q, k, v, causal=1, stream=s[0])
        y = sa.sparse_attn_forward_masked(t, kc, vc, stream=s[1])
        z = sa.sparse_attn_forward_masked(t, kc, vc, stream=s[0])
        torch.cuda.synchronize()
        for got, want in ((x, a), (y, b), (z, b)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# few rows over many keys: each lane quarter takes a quarter of them, and the runs are joined
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq", [(1, 1, 1), (4, 2, 1), (32, 1, 1), (3, 1, 10), (5, 1, 6), (6, 2, 11)])
@pytest.mark.parametrize("kw", [{}, dict(causal=1), dict(cap=20.0), dict(bias=True, causal=1), dict(bias=True, cap=5.0)])
def test_few_rows(d, H, Hk, Nq, kw):
    q, k, v = tensors(2, H, Hk, Nq, 3001, d, seed=30 + H, sigma=3.0)
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["slopes"] = [2.0 ** -(2 + i % 8) for i in range(H)]
    check(*run(q, k, v, out_dtype=torch.float32, **kw), q, k, v, **kw)


@pytest.mark.parametrize("Nq", [1, 3])
@pytest.mark.parametrize("lengths", [[20000, 0, 1, 129, 15001], [0, 0, 0, 0, 0], [5, 20000, 20000, 3, 2], [-7, 2, 99999, 128, 0]])
def test_few_rows_over_ragged_lengths(Nq, lengths):
    q, k, v = tensors(5, 8, 2, Nq, 20000, 64, seed=31)
    for b, n in enumerate(lengths):
        k[b, :, max(n, 0):] = float("nan")
        v[b, :, max(n, 0):] = float("nan")
    live = [min(max(n, 0), 20000) for n in lengths]
    check(*run(q, k, v, lengths=lengths, causal=1), q, k, v, lengths=live, causal=1)
    check(*run(q, k, v, lengths=lengths, cap=30.0), q, k, v, lengths=live, cap=30.0)


def test_few_rows_of_many_sequences_and_documents():
    g = np.random.default_rng(4)
    for B in (40, 76):
        lengths = [int(x) for x in g.integers(0, 4001, B)]
        q, k, v = tensors(B, 1, 1, 1, 4000, 64, seed=32)
        check(*run(q, k, v, lengths=lengths), q, k, v, lengths=lengths)
    docs = dict(docs_q=[[0, 2, 2, 9], [1, 1, 1, 8], [0, 3, 6, 9]], docs_k=[[0, 7000, 7001, 9000], [10, 20, 30, 9001],
                                                                          [0, 0, 4000, 4100]])
    q, k, v = tensors(3, 3, 1, 9, 9001, 128, seed=33)
    check(*run(q, k, v, causal=1, **docs), q, k, v, causal=1, **docs)
    check(*run(q, k, v, cap=9.0, **docs), q, k, v, cap=9.0, **docs)


@pytest.mark.parametrize("slopes", [None, [0.01, 0.02]])
def test_few_rows_late_maximum(slopes):
    q, k, v = tensors(1, 2, 1, 4, 5000, 128, seed=34)
    k[:, :, :100] *= 12  # tiles are taken from the last to the first
    k[:, :, 2500:2520] *= 6
    check(*run(q, k, v, slopes=slopes), q, k, v, slopes=slopes)
    check(*run(q, k, v, scale=-0.2), q, k, v, scale=-0.2)


def test_few_rows_streams_graphs_and_repeatability():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(3, 8, 2, 1, 20000, 128, seed=35)
    n = torch.tensor([20000, 1, 9000], dtype=torch.int32, device="cuda")
    want = sa.sparse_attn_forward_masked(q, k, v, lengths=n)
    other = sa.sparse_attn_forward_masked(q, k, v, lengths=n)
    assert torch.equal(want[0], other[0]) and torch.equal(want[1], other[1])
    out, lse = torch.empty_like(q), torch.empty(3, 8, 1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sparse_attn_forward_masked(q, k, v, lengths=n, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    n.copy_(torch.tensor([300, 20000, 0]))  # the captured call reads the lengths when it runs
    want = sa.sparse_attn_forward_masked(q, k, v, lengths=n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((out[2] == 0).all()) and bool((lse[2] == -float("inf")).all())


def test_output_over_the_queries():
    from video_dit_sparse_gb300 import binding as sa
    for H, Nq, Nk in ((4, 700, 900), (42, 515, 300), (8, 1, 4000)):
        q, k, v = tensors(2, H, 2, Nq, Nk, 128, seed=26)
        want, wl = sa.sparse_attn_forward_masked(q, k, v, causal=1)
        o, lse = sa.sparse_attn_forward_masked(q, k, v, causal=1, out=q)
        assert o is q and torch.equal(o, want) and torch.equal(lse, wl)
    qkv = tensors(2, 16, 1, 515, 1, 64, seed=27)[0].transpose(1, 2).contiguous().transpose(1, 2)
    q, k, v = qkv[:, :12], qkv[:, 12:14], qkv[:, 14:]
    want, _ = sa.sparse_attn_forward_masked(q, k, v, causal=1)
    rest = qkv[:, 12:].clone()
    sa.sparse_attn_forward_masked(q, k, v, causal=1, out=q)
    assert torch.equal(q, want) and torch.equal(qkv[:, 12:], rest)
    with pytest.raises(sa.SparseAttnError):
        sa.sparse_attn_forward_masked(k, k, v, out=k)


def test_few_rows_while_the_gpu_is_busy():
    """Blocks that start late or not at all: others take their runs over, and the table of runs is there all the same."""
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(4, 8, 2, 1, 20000, 64, seed=36)
    n = torch.tensor([20000, 3, 0, 11001], dtype=torch.int32, device="cuda")
    want = sa.sparse_attn_forward_masked(q, k, v, lengths=n)
    big = tensors(1, 12, 12, 2000, 4000, 128, seed=37)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(2):
            sa.sparse_attn_forward_masked(*big, stream=s[0])
        ws = torch.full((32 << 20,), 255, dtype=torch.uint8, device="cuda")  # (a table of -1 unless written)
        torch.cuda.current_stream().synchronize()
        o, lse = sa.sparse_attn_forward_masked(q, k, v, lengths=n, workspace=ws, stream=s[1])
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
