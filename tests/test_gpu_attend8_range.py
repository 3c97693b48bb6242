"""GPU checks of the attention over an 8-bit cache on each form that the sizes choose: every row width and block, heads that
are cut and joined, units that are split, ragged and empty entries in all of them, and both sides of every switch (16 rows of
a key head, 1024 tokens, 1024 entries).  Tolerances: the head of test_gpu_attend8.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attend8 import check, filled, rows, run

pytestmark = pytest.mark.gpu

RAGGED = [0, 1, 9999, 129, 128, 3, 2300, -5, 1333]


@pytest.mark.parametrize("d,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("H,Nq,causal", [(4, 1, 0), (4, 1, 1), (2, 8, 1), (6, 5, 3), (32, 1, 0)])
@pytest.mark.parametrize("Nk", [1025, 2300])
def test_cut_heads_of_ragged_entries(d, block, H, Nq, causal, Nk):
    """Few rows over heads that are cut: entries without keys, of one tile, and of more than a block's share."""
    c = filled(9, 2, Nk, d, block, seed=3, layout="bnhd")
    q = rows(9, H, Nq, d, 5, layout="bnhd")
    check(*run(q, c, causal=causal, lengths=RAGGED), q, c, causal=causal, lengths=RAGGED)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[0] * 9, [0] * 8 + [2300], [2300] + [0] * 8, [1] * 9])
def test_cut_heads_of_next_to_nothing(d, lengths):
    c = filled(9, 1, 2300, d, 64, seed=4)
    q = rows(9, 3, 2, d, 6)
    check(*run(q, c, causal=1, lengths=lengths), q, c, causal=1, lengths=lengths)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Nq", [(1, 1), (5, 3)])
def test_one_long_head_over_all_blocks(d, H, Nq):
    c = filled(1, 1, 33001, d, 16, seed=5)
    q = rows(1, H, Nq, d, 7)
    check(*run(q, c, causal=1), q, c, causal=1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Nq", [(1, 17), (3, 11), (2, 150), (1, 300)])
@pytest.mark.parametrize("Nk,causal", [(333, 0), (777, 1)])
def test_many_rows_of_every_width_and_block(d, block, H, Nq, Nk, causal):
    c = filled(1, 1, Nk, d, block, seed=8, spread=1.5)
    q = rows(1, H, Nq, d, 9)
    check(*run(q, c, causal=causal, out_dtype=torch.float32), q, c, causal=causal)


@pytest.mark.parametrize("d,block", [(64, 32), (128, 16)])
@pytest.mark.parametrize("Nq,causal", [(40, 0), (40, 1), (300, 7), (300, 880)])
def test_many_rows_of_ragged_entries(d, block, Nq, causal):
    lengths = [0, 1, 129, 700, 9999, -5]
    c = filled(6, 1, 700, d, block, seed=10, layout="bnhd")
    q = rows(6, 2, Nq, d, 11, layout="bnhd")
    check(*run(q, c, causal=causal, lengths=lengths), q, c, causal=causal, lengths=lengths)


@pytest.mark.parametrize("d,block", [(64, 32), (64, 128), (128, 16)])
@pytest.mark.parametrize("Nq", [40, 300])
def test_split_units_of_ragged_entries(d, block, Nq):
    lengths = [5001, 0, 2999, 100]
    c = filled(4, 2, 5001, d, block, seed=12)
    q = rows(4, 2, Nq, d, 13)
    check(*run(q, c, causal=1, lengths=lengths), q, c, causal=1, lengths=lengths)
    check(*run(q, c, out_dtype=torch.float32), q, c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Nq", [(16, 1), (17, 1), (4, 4), (1, 16), (1, 17), (128, 1)])
@pytest.mark.parametrize("Nk", [1024, 1025])
def test_both_sides_of_the_switches(d, H, Nq, Nk):
    c = filled(2, 1, Nk, d, 64, seed=14)
    q = rows(2, H, Nq, d, 15)
    check(*run(q, c, causal=1, lengths=[Nk, 500]), q, c, causal=1, lengths=[Nk, 500])


@pytest.mark.parametrize("B", [1024, 1025])
@pytest.mark.parametrize("Nk", [130, 1100])
def test_more_entries_than_the_table_holds(B, Nk):
    lengths = np.random.default_rng(B).integers(0, Nk + 1, size=B).tolist()
    c = filled(B, 1, Nk, 64, 64, seed=16)
    q = rows(B, 2, 1, 64, 17)
    check(*run(q, c, causal=1, lengths=lengths), q, c, causal=1, lengths=lengths)
