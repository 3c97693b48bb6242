"""GPU check of the 8-bit cache's reading into an output of more than 2^32 pieces of 16 codes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_reading_more_than_2_29_tokens():
    """d = 128: a token has eight pieces.  The cache is small: tokens outside it are zeros."""
    from video_dit_sparse_gb300 import binding as sa
    n, N, d = 2 ** 29 + 1000, 300, 128
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * n * d + (16 << 30):
        pytest.skip("137 GB of output")
    c = sa.sparse_attn_cache8(1, 1, N, d, block=16)
    x = torch.randn(1, 1, N, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    sa.sparse_attn_cache8_append(c, x, x, 0)
    out = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
    ends = (slice(0, 5000), slice(2 ** 28 - 5000, 2 ** 28 + 5000), slice(n - 5000, n - N), slice(n - N, n))
    for s in ends:
        out[:, :, s] = 7.0
    sa.sparse_attn_cache8_read(c, N - n, n, out=(out, None))
    want = sa.sparse_attn_cache8_read(c, 0, N)[0]
    ok = [not bool(out[:, :, s].any()) for s in ends[:3]] + [torch.equal(out[:, :, ends[3]], want)]
    del out
    torch.cuda.empty_cache()
    assert ok == [True] * 4
