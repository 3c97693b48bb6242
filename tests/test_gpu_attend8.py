"""GPU checks of the attention over an 8-bit cache against the 64-bit form on the values that the cache holds.

Tolerances.  Products of codes are exact in fp32; a score is off by the sum's e1 = d 2^-23 a (a: the largest
scale * sum |q k| of the head) and by the query row's two terms, e2 = 2^-17 scale max |q| sum |k|.  Weights reach the
second product with at least ten bits (2^-10 of each; what lies below 2^-28 of the row's largest may be lost), so
    |o - want| <= (2^-10 + 2 e + 2^-16) 1.01 (sum p |v| + |want|) + 2^-28 sum |v| + the output's own rounding,
    |lse - want| <= e + 2^-20 (1 + |want|)."""
import numpy as np
import pytest
import torch

from oracle import cache8_ops as P

pytestmark = pytest.mark.gpu


def rows(B, H, N, d, seed, layout="bhnd", sigma=1.5, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, H, N, d) if layout == "bhnd" else (B, N, H, d), generator=g) * sigma + mean).to(torch.bfloat16).cuda()
    return x if layout == "bhnd" else x.transpose(1, 2)


def filled(B, H, N, d, block, seed, layout="bhnd", spread=1.0):
    """A cache of N tokens of different size, written by the library itself."""
    from video_dit_sparse_gb300 import binding as sa
    c = sa.sparse_attn_cache8(B, H, N, d, block=block)
    if layout == "bnhd":
        k, v = (torch.zeros(B, N, H, d, dtype=torch.float8_e4m3fn, device="cuda").transpose(1, 2) for _ in range(2))
        c = c._replace(k=k, v=v)
    g = torch.Generator().manual_seed(seed + 1)
    loud = torch.exp(spread * torch.randn(B, H, N, 1, generator=g)).to(torch.bfloat16).cuda()
    sa.sparse_attn_cache8_append(c, rows(B, H, N, d, seed + 2, sigma=1.0, mean=0.3), rows(B, H, N, d, seed + 3, sigma=1.0) * loud, 0)
    return c


def held(c):
    """(k, v) [B, H, N, d] as float64 values."""
    out = []
    for codes, scales in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes, scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
        out.append(np.stack([np.stack([P.values(codes[b, h], scales[b, h], c.block) for h in range(codes.shape[1])])
                             for b in range(codes.shape[0])]))
    return out


def check(o, lse, q, c, *, scale=None, causal=0, lengths=None, kv=None):
    B, H, Nq, d = q.shape
    Hk, Nk = c.k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    k, v = held(c) if kv is None else kv
    q = q.double().cpu().numpy()
    eps = torch.finfo(o.dtype).eps / 2
    got, glse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        n = Nk if lengths is None else min(max(int(lengths[b]), 0), Nk)
        hi = P.row_ends(Nq, n, causal)
        for h in range(H):
            hk = h // (H // Hk)
            want, wlse, pv, a = P.attention(q[b, h], k[b, hk], v[b, hk], scale, hi)
            ks = np.abs(k[b, hk, :max(hi.max(), 0)])
            e = d * 2.0 ** -23 * a + 2.0 ** -17 * abs(scale) * np.abs(q[b, h]).max() * ks.sum(-1).max(initial=0.0)
            lost = 2.0 ** -28 * np.abs(v[b, hk, :max(hi.max(), 0)]).sum(0)
            tol = (2.0 ** -10 + 2 * e + 2.0 ** -16) * 1.01 * (pv + np.abs(want)) + lost + eps * np.abs(want)
            err = np.abs(got[b, h] - want)
            assert (err <= tol).all(), (b, h, float((err - tol).max()), np.argwhere(~(err <= tol))[:4], e)
            none = np.isinf(wlse)
            assert np.array_equal(glse[b, h] == -np.inf, none)
            assert (got[b, h][none] == 0).all()
            lerr = np.abs(glse[b, h][~none] - wlse[~none])
            assert (lerr <= (e + 2.0 ** -20 * (1 + np.abs(wlse[~none])))).all(), (float(lerr.max()), e)


def run(q, c, **kw):
    from video_dit_sparse_gb300 import binding as sa
    if kw.get("lengths") is not None:
        kw["lengths"] = torch.tensor(kw["lengths"], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sa.sparse_attn_forward_cache8(q, c, status=status, **kw)
    assert int(status) == 0
    return o, lse


# rows of a key head: one, a few, all of each kernel's sizes; keys: one to several tiles, odd
FEW = [(1, 1, 1, 1), (2, 2, 1, 129), (8, 1, 1, 640), (3, 1, 5, 257), (16, 1, 1, 1000), (2, 1, 16, 128), (8, 2, 4, 513),
       (4, 4, 32, 300), (32, 1, 1, 77)]


@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("H,Hk,Nq,Nk", FEW)
@pytest.mark.parametrize("causal", [0, 1, 97])
def test_few_rows(d, block, H, Hk, Nq, Nk, causal):
    c = filled(2, Hk, Nk, d, block, seed=Nq + Nk)
    q = rows(2, H, Nq, d, 7 * Nq + Nk)
    check(*run(q, c, causal=causal), q, c, causal=causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Nq,causal", [(4, 1, 0), (4, 1, 1), (2, 7, 1), (6, 5, 3)])
def test_ragged_lengths(d, H, Nq, causal):
    """More sequences than blocks share evenly; none, one, a part, all and more than all of the cache."""
    B, Hk, Nk = 9, 2, 700
    lengths = [0, 1, 700, 129, 128, 3, 9999, -5, 333]
    c = filled(B, Hk, Nk, d, 32, seed=3, layout="bnhd")
    q = rows(B, H, Nq, d, 5, layout="bnhd")
    check(*run(q, c, causal=causal, lengths=lengths), q, c, causal=causal, lengths=lengths)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 4])
def test_lse_of_one_key_keeps_its_own_precision(d, Nq):
    """One key, one column that is not 0: lse is the score, however small.  Its roundings (the scale's, its product with
    log2 e, the score's, its product with ln 2) are 2^-24 of it each, the two constants' 2^-25: below 2^-21 together."""
    from video_dit_sparse_gb300 import binding as sa
    c = sa.sparse_attn_cache8(1, 2, 1, d, block=16)
    k = torch.zeros(1, 2, 1, d)
    k[..., 5] = 0.7
    sa.sparse_attn_cache8_append(c, k.to(torch.bfloat16).cuda(), rows(1, 2, 1, d, 1), 0)
    q = torch.zeros(1, 4, Nq, d)
    q[..., 5] = torch.tensor([0.01, -0.3, 1.1, 40.0])[None, :, None] * torch.linspace(1, 1.7, Nq)
    q = q.to(torch.bfloat16).cuda()
    _, lse = run(q, c, scale=0.3)
    want = q[..., 5].double().cpu().numpy() * held(c)[0][:, :, 0, 5].repeat(2, 1)[..., None] * 0.3
    assert (np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -21 * np.abs(want)).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 4])
def test_lse_of_one_key_beside_a_large_query_value(d, Nq):
    """The column that counts is 2^-10 to 2^-16 of the row's largest, whose key is 0: the row's two terms are off by
    2^-22 of that largest, what is left as in the test above."""
    from video_dit_sparse_gb300 import binding as sa
    c = sa.sparse_attn_cache8(1, 2, 1, d, block=16)
    k = torch.zeros(1, 2, 1, d)
    k[..., 5] = 0.7
    sa.sparse_attn_cache8_append(c, k.to(torch.bfloat16).cuda(), rows(1, 2, 1, d, 1), 0)
    q = torch.zeros(1, 4, Nq, d)
    q[..., 9] = 1.9
    q[..., 5] = torch.tensor([1.3e-3, -7.7e-4, 2.3e-4, 3.1e-5])[None, :, None] * torch.linspace(1, 1.7, Nq)
    q = q.to(torch.bfloat16).cuda()
    _, lse = run(q, c, scale=0.3)
    held_k = held(c)[0][:, :, 0, 5].repeat(2, 1)[..., None]
    want = q[..., 5].double().cpu().numpy() * held_k * 0.3
    assert (np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -21 * np.abs(want) + 2.0 ** -22 * 1.9 * held_k * 0.3).all()


@pytest.mark.parametrize("H,Nq", [(2, 1), (2, 40)])
def test_long_caches_many_splits(H, Nq):
    c = filled(1, 2, 33000, 128, 128, seed=4)
    q = rows(1, H, Nq, 128, 6)
    check(*run(q, c, causal=1), q, c, causal=1)
    check(*run(q, c, causal=1, out_dtype=torch.float32, scale=-0.11), q, c, causal=1, scale=-0.11)


@pytest.mark.parametrize("Nq", [1, 6, 150])
def test_rising_scores_move_the_reference(Nq):
    """Keys in order of their product with the query, over more than fp16's and e5m2's range, both ways."""
    from video_dit_sparse_gb300 import binding as sa
    d, N = 128, 1500
    for sign in (1.0, -1.0):
        ramp = torch.linspace(0, 6, N)[None, None, :, None] * sign
        k = (ramp * torch.ones(1, 1, N, d) + 0.05 * torch.randn(1, 1, N, d, generator=torch.Generator().manual_seed(1)))
        c = sa.sparse_attn_cache8(1, 1, N, d, block=64)
        sa.sparse_attn_cache8_append(c, k.to(torch.bfloat16).cuda(), rows(1, 1, N, d, 2), 0)
        q = torch.ones(1, 2, Nq, d, dtype=torch.bfloat16, device="cuda") * torch.tensor([1.0, -0.7], device="cuda")[None, :, None, None].bfloat16()
        check(*run(q, c, causal=1), q, c, causal=1)


@pytest.mark.parametrize("Nq", [1, 3, 140])
def test_value_scales_far_apart(Nq):
    """Blocks of values 2^40 larger and smaller than their neighbours."""
    from video_dit_sparse_gb300 import binding as sa
    c = filled(1, 2, 500, 64, 16, seed=8)
    c.v_scale.mul_(2.0 ** torch.randint(-40, 41, c.v_scale.shape, generator=torch.Generator().manual_seed(2)).cuda())
    q = rows(1, 4, Nq, 64, 9)
    check(*run(q, c, out_dtype=torch.float32), q, c)
    c.k_scale.mul_(0.37)  # not powers of two
    c.v_scale.mul_(0.37)
    o, lse = run(q, c, out_dtype=torch.float32)
    check(o, lse, q, c)
    low = sa.sparse_attn_forward_cache8(q, c)[0]
    assert torch.equal(low, o.to(torch.bfloat16))


@pytest.mark.parametrize("Nq", [1, 5, 40, 300])
def test_what_a_row_does_not_see(Nq):
    """NaN codes and bad scales behind the sequence, and in the keys that only later rows see, change nothing."""
    from video_dit_sparse_gb300 import binding as sa
    B, H, Hk, N, d = 2, 2, 1, 700, 128
    n = [430, 561]
    c = filled(B, Hk, N, d, 64, seed=11)
    q = rows(B, H, Nq, d, 12)
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    want, wlse = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    k, v = c.k.view(torch.uint8), c.v.view(torch.uint8)
    for b in range(B):
        k[b, :, n[b]:], v[b, :, n[b]:] = 0x7F, 0xFF
    c.k_scale[:, :, 9:], c.v_scale[:, :, 9:] = float("nan"), float("inf")
    got, lse = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    assert torch.equal(got, want) and torch.equal(lse, wlse)
    # the last token's value: a NaN in two of its columns reaches the row that sees it, in these columns alone
    for b in range(B):
        v[b, 0, n[b] - 1, 5] = 0x7F
        v[b, 0, n[b] - 1, 77] = 0xFF
    got, lse = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    bad = torch.isnan(got)
    assert bool(bad[:, :, -1, [5, 77]].all()) and int(bad.sum()) == 2 * B * H
    assert torch.equal(lse, wlse) and torch.equal(got[:, :, :-1], want[:, :, :-1])
    keep = [i for i in range(d) if i not in (5, 77)]
    # (a column's sum does not go by the other columns)
    assert torch.equal(got[:, :, -1][..., keep], want[:, :, -1][..., keep])
    # the last token's key: NaN for the row that sees it, whole
    for b in range(B):
        k[b, 0, n[b] - 1, 9] = 0x7F
    got, lse = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    assert bool(torch.isnan(got[:, :, -1]).all()) and bool(torch.isnan(lse[:, :, -1]).all())
    assert torch.equal(got[:, :, :-1], want[:, :, :-1]) and torch.equal(lse[:, :, :-1], wlse[:, :, :-1])


@pytest.mark.parametrize("Nq", [1, 5, 200])
def test_empty_blocks_are_zeros(Nq):
    """A block whose scale is no positive finite number holds zeros, whatever its codes: its keys score 0."""
    c = filled(1, 1, 512, 128, 128, seed=13)
    c.k.view(torch.uint8)[0, 0, 128:256] = 0x7F
    c.v.view(torch.uint8)[0, 0, 128:256] = 0x7F
    c.k_scale[0, 0, 1], c.v_scale[0, 0, 1] = 0.0, float("nan")
    q = rows(1, 2, Nq, 128, 14)
    kv = held(c)
    assert (kv[0][0, 0, 128:256] == 0).all()
    check(*run(q, c), q, c, kv=kv)


@pytest.mark.parametrize("Nq", [1, 20, 300])
def test_query_rows_of_any_size(Nq):
    """Rows of zeros, of tiny and of huge values; what is not finite stays in its row."""
    c = filled(1, 1, 300, 128, 64, seed=15)
    q = rows(1, 1, Nq, 128, 16)
    q[0, 0, 0] = 0
    if Nq > 1:
        q[0, 0, 1] *= 2.0 ** -120
        q[0, 0, 2, 3:] = 2.0 ** -130
        q[0, 0, 3, 1:] *= 2.0 ** -9
    check(*run(q, c), q, c)
    q[0, 0, 0, 4] = float("inf")
    o, lse = run(q, c)
    assert bool(torch.isnan(o[0, 0, 0]).all()) and bool(torch.isnan(lse[0, 0, 0]))
    assert bool(torch.isfinite(o[0, 0, 1:]).all())


@pytest.mark.parametrize("Nq", [1, 9, 260])
def test_strides_in_place_streams_and_graphs(Nq):
    from video_dit_sparse_gb300 import binding as sa
    B, H, Hk, N, d = 2, 4, 2, 1030, 128
    big = filled(B, Hk + 1, N, d, 64, seed=17, layout="bnhd")
    c = sa.Cache8(big.k[:, 1:], big.v[:, 1:], big.k_scale[:, 1:], big.v_scale[:, 1:], 64)
    buf = rows(B, H + 3, Nq, d, 18, layout="bnhd")
    q = buf[:, 1:H + 1]
    want, wlse = run(q, c, causal=1)
    check(want, wlse, q, c, causal=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = sa.sparse_attn_forward_cache8(q, c, causal=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    lengths = torch.tensor([N, N], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    lengths.copy_(torch.tensor([77, 901]))
    graph.replay()
    o2, lse2 = sa.sparse_attn_forward_cache8(q, c, causal=1, lengths=lengths)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(o, lse, q, c, causal=1, lengths=[77, 901])
    inplace, _ = sa.sparse_attn_forward_cache8(q, c, causal=1, out=q, lse=False)
    assert inplace.data_ptr() == q.data_ptr() and torch.equal(q, want)


@pytest.mark.parametrize("Nq", [1, 70])
def test_offsets_past_32_bits(Nq):
    """Keys behind the first 2^32 codes of a head."""
    from video_dit_sparse_gb300 import binding as sa
    N, d = 2 ** 25 + 2 ** 10, 128
    c = sa.sparse_attn_cache8(1, 1, N, d, block=128)
    at = N - 300
    sa.sparse_attn_cache8_append(c, rows(1, 1, 300, d, 20) + 4.0, rows(1, 1, 300, d, 21), at)
    q = rows(1, 1, Nq, d, 22).abs() * 4 + 2  # scores far above the empty keys' 0
    o, lse = run(q, c)
    small = sa.sparse_attn_cache8(1, 1, 300, d, block=128)
    k, v = sa.sparse_attn_cache8_read(c, at, 300)
    sa.sparse_attn_cache8_append(small, k, v, 0)
    kv = [x.double().cpu().numpy() for x in (k, v)]
    check(o, lse, q, small, kv=kv)  # 2^25 weights of e^0 beside e^50 and more: below 2^-40
