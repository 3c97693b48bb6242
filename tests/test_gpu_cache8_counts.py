"""Token numbers that do not fit the 32 bits of the entry points are refused by the binding, not taken for others."""
import pytest
import torch


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 1, 2 ** 32 + 5])
def test_more_tokens_than_32_bits(n):
    from video_dit_sparse_gb300 import binding as sa
    c = sa.sparse_attn_cache8(1, 1, 64, 64, block=16)
    x = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(1, 1, n, 64)  # one row repeated
    with pytest.raises(ValueError):
        sa.sparse_attn_cache8_append(c, x, x, 0)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache8_read(c, 0, n, out=(x, None))
    assert not bool(c.k_scale.any())


def test_counts_fit_32_bits():
    from video_dit_sparse_gb300 import build
    build.build()
    from video_dit_sparse_gb300 import binding as sa
    assert sa._count(0) == 0 and sa._count(2 ** 31 - 1) == 2 ** 31 - 1 and sa._count(-1) == -1
    for n in (2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            sa._count(n)


def test_tokens_are_whole_numbers():
    """A first token of 2.5 is not taken for 2."""
    from video_dit_sparse_gb300 import build
    build.build()
    from video_dit_sparse_gb300 import binding as sa
    assert sa._tokens(3.0, "start", 0, 1) == (0, 3)
    for at in (2.5, -0.5, "4", float("nan")):
        with pytest.raises(ValueError):
            sa._tokens(at, "start", 0, 1)
