"""GPU checks of the attention over an 8-bit cache whose values' scales are the smallest that the cache makes (2^-126):
the outputs are normal numbers, and keep the tolerances at the head of test_gpu_attend8.py."""
import pytest
import torch

from tests.test_gpu_attend8 import check, filled, rows, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 12, 40, 300])
@pytest.mark.parametrize("N,e", [(900, -126), (6000, -118), (6000, -126)])
def test_smallest_scales(d, Nq, N, e):
    """Values of one sign, so that an output is their mean's size, 2^5 of the scale and more; scores of 0, which are exact,
    so that every key weighs the same and the row's sum is as large as it gets."""
    c = filled(1, 1, N, d, 128, seed=3, spread=0.0)
    c.v.view(torch.uint8).bitwise_and_(0x7F)
    c.v_scale.fill_(2.0 ** e)
    q = rows(1, 1, Nq, d, 5)
    check(*run(q, c, out_dtype=torch.float32), q, c)
    q.zero_()
    check(*run(q, c, out_dtype=torch.float32), q, c)
