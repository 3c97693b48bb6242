"""GPU checks of what is not finite: a query that is not a number makes its row's output and lse none, on every path.
Other rows are compared with the 64-bit form within test_gpu_masked's tolerances."""
import pytest
import torch

from tests.test_gpu_masked import check, run, tensors

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.mark.parametrize("H,Hk,Nq,Nk,kw", [
    (4, 2, 1, 20000, {}), (4, 2, 1, 20000, dict(lengths=[20000, 15000])), (3, 1, 40, 8000, {}), (1, 1, 700, 900, {}),
    (8, 2, 17, 640, dict(causal=1))])
def test_a_query_that_is_not_a_number_comes_out(H, Hk, Nq, Nk, kw):
    """Whole, and joined from partial results that are all no numbers: not a row that saw nothing."""
    q, k, v = tensors(2, H, Hk, Nq, Nk, 128, seed=62)
    clean, cl = run(q, k, v, **kw)
    q0 = q.clone()
    q[1, 0, Nq // 2, 3] = NAN
    o, lse = run(q, k, v, **kw)
    assert bool(torch.isnan(o[1, 0, Nq // 2]).all()) and bool(torch.isnan(lse[1, 0, Nq // 2]))
    o[1, 0, Nq // 2], lse[1, 0, Nq // 2] = clean[1, 0, Nq // 2], cl[1, 0, Nq // 2]
    check(o, lse, q0, k, v, **kw)
