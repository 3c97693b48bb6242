"""GPU checks of the 8-bit cache's writing and reading against the 64-bit forms: codes, scales and values are the same,
bit for bit (scales are powers of two, so x / scale is exact and only the one rounding to a code is left)."""
import numpy as np
import pytest
import torch

from oracle import cache8_ops as P

pytestmark = pytest.mark.gpu


def tokens(B, H, n, d, seed, layout="bhnd", spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, H, n, d) if layout == "bhnd" else (B, n, H, d), generator=g)
    x = x * torch.exp(spread * torch.randn(x.shape[:-1] + (1,), generator=g))  # tokens of different size
    x = x.to(torch.bfloat16).cuda()
    return x if layout == "bhnd" else x.transpose(1, 2)


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


class Mirror:
    """A cache on the GPU and what it should hold."""

    def __init__(self, B, H, N, d, block, layout="bhnd"):
        from video_dit_sparse_gb300 import binding as sa
        self.sa, self.block = sa, block
        self.c = sa.sparse_attn_cache8(B, H, N, d, block=block)
        if layout == "bnhd":
            k, v = (torch.zeros(B, N, H, d, dtype=torch.float8_e4m3fn, device="cuda").transpose(1, 2) for _ in range(2))
            self.c = self.c._replace(k=k, v=v)
        self.codes = [bits(self.c.k).copy(), bits(self.c.v).copy()]
        self.scales = [np.zeros((B, H, -(-N // block))) for _ in range(2)]

    def append(self, k, v, start, counts=None, **kw):
        B, H, n, _ = k.shape
        at = [start] * B if isinstance(start, int) else start
        dev = start if isinstance(start, int) else torch.tensor(start, dtype=torch.int32, device="cuda")
        cn = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        assert self.sa.sparse_attn_cache8_append(self.c, k, v, dev, counts=cn, **kw) is self.c
        for i, x in enumerate((k, v)):
            x = x.double().cpu().numpy()
            for b in range(B):
                m = n if counts is None else min(max(counts[b], 0), n)
                for h in range(H):
                    self.codes[i][b, h], self.scales[i][b, h] = P.append(self.codes[i][b, h], self.scales[i][b, h], x[b, h],
                                                                         at[b], m, self.block)

    def check(self):
        for i, (codes, scales) in enumerate(((self.c.k, self.c.k_scale), (self.c.v, self.c.v_scale))):
            assert np.array_equal(scales.double().cpu().numpy(), self.scales[i])
            got = bits(codes)
            # a NaN keeps no sign
            same = (got == self.codes[i]) | (((got & 127) == 127) & ((self.codes[i] & 127) == 127))
            assert same.all(), np.argwhere(~same)[:4]

    def values(self, i, b, first, n):
        """Tokens first .. first + n - 1 of the i-th tensor, entry b: [H, n, d]."""
        H, N, d = self.codes[i].shape[1:]
        out = np.zeros((H, n, d))
        for h in range(H):
            x = P.values(self.codes[i][b, h], self.scales[i][b, h], self.block)
            for t in range(n):
                if 0 <= first + t < N:
                    out[h, t] = x[first + t]
        return out


def test_forms():
    """The codes' table and its rounding against torch's own type."""
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * torch.exp(3 * torch.randn(4096))
    x = x.clamp(-448, 448)
    assert np.array_equal(P.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    every = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(P.decode(every.numpy()), every.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    assert P.scale_for(448.0) == 1 and P.scale_for(449.0) == 2 and P.scale_for(2.0 ** -140) == 2.0 ** -126


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d,layout", [(64, "bnhd"), (128, "bhnd")])
@pytest.mark.parametrize("N,steps", [(1, (1,)), (300, (1, 16, 1, 1, 37, 128, 1)), (257, (257,)), (640, (128, 512))])
def test_filling_in_order(block, d, layout, N, steps):
    m = Mirror(2, 3, N, d, block, layout)
    at = 0
    for i, n in enumerate(steps):
        m.append(tokens(2, 3, n, d, 10 + i, layout), tokens(2, 3, n, d, 20 + i, layout, spread=2.0), at)
        m.check()
        at += n


@pytest.mark.parametrize("block", [16, 64])
def test_ragged_starts_and_counts(block):
    m = Mirror(4, 2, 200, 64, block)
    m.append(tokens(4, 2, 200, 64, 1), tokens(4, 2, 200, 64, 2), 0)
    # before the cache, across its end, none, all; a count above n is n
    m.append(tokens(4, 2, 50, 64, 3, spread=2.0), tokens(4, 2, 50, 64, 4, spread=2.0), [-20, 180, 77, 33], [50, 50, 0, 99])
    m.check()
    m.append(tokens(4, 2, 50, 64, 5), tokens(4, 2, 50, 64, 6), [-60, 200, 2 ** 31 - 1, -2 ** 31], [50, -3, 50, 50])
    m.check()  # nothing of these lies in the cache


def test_rewriting_whole_blocks_forgets_their_scale():
    m = Mirror(1, 2, 256, 128, 128)
    m.append(tokens(1, 2, 256, 128, 1) * 1000, tokens(1, 2, 256, 128, 2) * 1000, 0)
    m.append(tokens(1, 2, 128, 128, 3), tokens(1, 2, 128, 128, 4), 128)
    m.check()
    assert float(m.c.k_scale[0, 0, 1]) < float(m.c.k_scale[0, 0, 0]) / 100
    m.append(tokens(1, 2, 1, 128, 5), tokens(1, 2, 1, 128, 6), 5)  # a part keeps the larger scale
    m.check()


def test_zeros_extremes_and_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    m = Mirror(1, 1, 96, 64, 16)
    k, v = torch.zeros(2, 1, 1, 96, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 17, 3] = inf            # the only value of its block
    k[0, 0, 33, :4] = torch.tensor([1.0, nan, -inf, 448.0])
    k[0, 0, 49, 0] = 3.3e38
    k[0, 0, 50, 0] = 1e-38
    k[0, 0, 65, 0] = 9.2e-41        # below the least scale's steps
    v[0, 0, :, :] = 2.0 ** -133     # the smallest bf16
    v[0, 0, 40] = -0.0
    m.append(k, v, 0)
    m.check()
    assert m.scales[0][0, 0].tolist() == [0.0, 2.0 ** -126, 1.0, 2.0 ** 120, 2.0 ** -126, 0.0]
    m.append(tokens(1, 1, 1, 64, 1), tokens(1, 1, 1, 64, 2), 18)  # the NaN beside it stays one
    m.check()
    got, _ = m.sa.sparse_attn_cache8_read(m.c, 0, 96, out_dtype=torch.float32)
    with np.errstate(over="ignore"):  # (3.3e38 is held as 256 2^120 = 2^128: beyond fp32, whose rounding of it is infinite)
        want = m.values(0, 0, 0, 96).astype(np.float32)
    assert np.array_equal(got.cpu().numpy()[0], want, equal_nan=True)
    assert torch.isnan(got[0, 0, 17, 3]) and torch.isnan(got[0, 0, 33, 1])


def test_scales_of_other_makers():
    """A cache filled elsewhere: scales that are no powers of two, empty blocks with any code."""
    from video_dit_sparse_gb300 import binding as sa
    g = torch.Generator().manual_seed(7)
    codes = torch.randint(0, 256, (1, 2, 64, 64), generator=g, dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0
    scale = torch.tensor([[[0.37, 0.0, -1.0, float("nan")], [1e-3, float("inf"), 5e30, 0.1]]])
    c = sa.Cache8(codes.cuda(), codes.cuda(), scale.cuda(), scale.cuda(), 16)
    got, _ = sa.sparse_attn_cache8_read(c, 0, 64, out_dtype=torch.float32)
    low, _ = sa.sparse_attn_cache8_read(c, 0, 64)
    s64 = scale.double().numpy()
    for h in range(2):
        want = P.values(codes[0, h].numpy(), s64[0, h], 16)
        assert np.array_equal(got[0, h].cpu().numpy(), want.astype(np.float32))  # one fp32 product
        assert torch.equal(low[0, h], got[0, h].to(torch.bfloat16))
    x = tokens(1, 2, 1, 64, 3, spread=0.0) * 0.01
    sa.sparse_attn_cache8_append(c, x, x, 3)
    assert torch.equal(c.k_scale[0, 0].cpu()[0], scale[0, 0, 0])  # large enough as it is
    want = P.encode(np.clip(x[0, 0, 0].float().cpu().numpy() / np.float32(0.37), -448, 448))
    assert np.array_equal(c.k[0, 0, 3].cpu().numpy(), want)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,d,layout", [(16, 64, "bhnd"), (128, 128, "bnhd")])
def test_reading(out_dtype, block, d, layout):
    m = Mirror(3, 2, 333, d, block, layout)
    m.append(tokens(3, 2, 333, d, 1, layout), tokens(3, 2, 333, d, 2, layout, spread=2.0), 0)
    first = [0, 300, -5]
    dev = torch.tensor(first, dtype=torch.int32, device="cuda")
    k, v = m.sa.sparse_attn_cache8_read(m.c, dev, 40, out_dtype=out_dtype)
    assert k.dtype is out_dtype
    for b in range(3):
        for i, t in enumerate((k, v)):
            assert np.array_equal(t[b].double().cpu().numpy(), m.values(i, b, first[b], 40))  # powers of two: exact
    out = torch.full((3, 40, 2, d), 7.0, dtype=out_dtype, device="cuda").transpose(1, 2)
    a, none = m.sa.sparse_attn_cache8_read(m.c, dev, 40, out=(None, out))
    assert a is None and none is out and torch.equal(out, v)


def test_streams_slices_graphs_and_far_offsets():
    from video_dit_sparse_gb300 import binding as sa
    big = sa.sparse_attn_cache8(2, 2, 2 ** 24 + 256, 128, block=128)  # 2^32 codes and more a batch entry
    c = sa.Cache8(big.k[:, 1:], big.v[:, 1:], big.k_scale[:, 1:], big.v_scale[:, 1:], 128)  # a slice of the heads
    k, v = tokens(2, 1, 130, 128, 1), tokens(2, 1, 130, 128, 2)
    at = torch.full((2,), 2 ** 24 + 60, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sa.sparse_attn_cache8_append(c, k, v, at, stream=side)
    a, b = sa.sparse_attn_cache8_read(c, at, 130, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    small = sa.sparse_attn_cache8(2, 1, 256, 128, block=128)
    sa.sparse_attn_cache8_append(small, k, v, 60)
    x, y = sa.sparse_attn_cache8_read(small, 60, 130)
    assert torch.equal(a, x) and torch.equal(b, y) and bool((a != 0).any())
    assert int(big.k.view(torch.uint8)[:, 0].max()) == 0 and int(big.k_scale[:, 0].count_nonzero()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sparse_attn_cache8_append(c, k, v, at)
        a, b = sa.sparse_attn_cache8_read(c, at, 130)
    at.fill_(1000)
    k.copy_(tokens(2, 1, 130, 128, 9))
    graph.replay()
    empty = sa.sparse_attn_cache8(2, 1, 2048, 128, block=128)
    sa.sparse_attn_cache8_append(empty, k, v, 1000)
    assert torch.equal(a, sa.sparse_attn_cache8_read(empty, 1000, 130)[0])
