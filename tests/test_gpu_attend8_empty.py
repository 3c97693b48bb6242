"""GPU checks of the attention over an 8-bit cache where value blocks are empty, and where values are small.

An empty block's keys weigh in a row's sum and add nothing to its output, so they must not cost the others' weights
digits: the tolerances are those at the head of test_gpu_attend8.py, with values of one size, so that sum |v| says nothing
that sum p |v| does not."""
import numpy as np
import pytest
import torch

from oracle import cache8_ops as P
from tests.test_gpu_attend8 import check, filled, held, rows, run

pytestmark = pytest.mark.gpu

F32 = torch.float32


def quiet(c, e, empty):
    """The cache's values 2^e times theirs, with the first `empty` blocks empty (any code, among them NaN)."""
    c.v_scale.copy_(c.v_scale.amax() * 2.0 ** e)
    c.v_scale[:, :, :empty] = 0.0
    c.v.view(torch.uint8)[:, :, :empty * c.block:7] = 0x7F
    return c


@pytest.mark.parametrize("Nq", [1, 5, 40, 300])
@pytest.mark.parametrize("d,block,empty", [(64, 16, 1), (64, 128, 1), (128, 32, 4), (128, 16, 21), (64, 64, 5), (128, 128, 3)])
@pytest.mark.parametrize("e", [-12, -24, -30, -60, -105])
def test_values_behind_empty_blocks_keep_their_digits(Nq, d, block, empty, e):
    """One empty block, a tile of them, several tiles of them, ahead of values of 2^e."""
    c = quiet(filled(1, 2, 701, d, block, seed=3, spread=0.0), e, empty)
    q = rows(1, 4, Nq, d, 5)
    check(*run(q, c, out_dtype=F32), q, c)
    check(*run(q, c, out_dtype=F32, causal=1), q, c, causal=1)


@pytest.mark.parametrize("Nq", [1, 40, 300])
def test_split_heads_behind_empty_blocks(Nq):
    """Heads that are cut, some parts of them of empty blocks alone, and entries of different length."""
    c = quiet(filled(3, 2, 5000, 64, 64, seed=7, spread=0.0), -40, 31)
    q = rows(3, 4, Nq, 64, 9)
    lengths = [5000, 1700, 2999]
    check(*run(q, c, out_dtype=F32, causal=97, lengths=lengths), q, c, causal=97, lengths=lengths)


@pytest.mark.parametrize("Nq", [2, 200])
def test_rows_that_see_empty_blocks_alone(Nq):
    """Keys and values empty: a row's lse is ln of its keys' number (no score is off), its output 0."""
    N = 128 + Nq - 1
    c = filled(1, 1, N, 128, 128, seed=11)
    c.k_scale[:, :, 0], c.v_scale[:, :, 0] = 0.0, 0.0
    q = rows(1, 2, Nq, 128, 12)
    o, lse = run(q, c, out_dtype=F32, causal=1)
    check(o, lse, q, c, causal=1)
    assert (np.abs(lse[:, :, 0].double().cpu().numpy() - np.log(128)) <= 2.0 ** -20).all() and not bool(o[:, :, 0].any())


@pytest.mark.parametrize("Nq", [1, 6, 40, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("down", [-60, -100])
def test_an_empty_block_between_loud_and_quiet_ones(Nq, d, down):
    """Rows that attend to quiet values (2^down) and, as much, to an empty block, but not to the loud block in front.

    The loud block's scores lie 80 below: its e^-80 of 2^0 is 2^-15 of what the quiet ones give (2^-100), or less.  So the
    output's size is the quiet values', and what may be lost of each weight is 2^-28 of the row's largest product."""
    from video_dit_sparse_gb300 import binding as sa
    N, block = 512, 128
    b = 40.0 / d ** 0.5  # a score of 40 either way
    k = torch.full((1, 1, N, d), b) + 0.05 * torch.randn(1, 1, N, d, generator=torch.Generator().manual_seed(1))
    k[:, :, :block] *= -1.0
    c = sa.sparse_attn_cache8(1, 1, N, d, block=block)
    sa.sparse_attn_cache8_append(c, k.to(torch.bfloat16).cuda(), rows(1, 1, N, d, 2, sigma=1.0), 0)
    c.v_scale[:, :, 1] = 0.0
    c.v_scale[:, :, 2:] *= 2.0 ** down
    q = torch.ones(1, 2, Nq, d, dtype=torch.bfloat16, device="cuda")
    o, lse = run(q, c, out_dtype=F32)
    hk, hv = held(c)
    want, wlse, pv, a = P.attention(q[0, 0].double().cpu().numpy(), hk[0, 0], hv[0, 0], d ** -0.5, P.row_ends(Nq, N, 0))
    e = d * 2.0 ** -23 * a + 2.0 ** -17 * d ** -0.5 * np.abs(hk[0, 0]).sum(-1).max()
    tol = (2.0 ** -10 + 2 * e + 2.0 ** -16) * 1.01 * (pv + np.abs(want)) + 2.0 ** -28 * np.abs(hv[0, 0, 2 * block:]).sum(0)
    for h in range(2):
        err = np.abs(o[0, h].double().cpu().numpy() - want)
        assert (err <= tol).all(), (float((err / tol).max()), float(np.abs(want).max()))
        assert (np.abs(lse[0, h].double().cpu().numpy() - wlse) <= e + 2.0 ** -20 * (1 + np.abs(wlse))).all()
