"""GPU checks of the masked forward where a distance bias meets documents: documents that start inside a key tile, rows
at and before their document's first key (more rows than keys, many heads on a key head), without a causal mask, with
frames and with prefixes, through every path (two tiles, one tile, split keys, few rows in every lane quarter).
Tolerances are those of test_gpu_masked."""
import pytest

from tests.test_gpu_masked import check, run, tensors

pytestmark = pytest.mark.gpu

# H, Hk, Nq, Nk, docs_q, docs_k
CASES = {
    "two tiles, more rows than keys": (1, 1, 300, 100, [0, 100, 300], [0, 40, 100]),
    "one tile, more rows than keys": (1, 1, 128, 60, [0, 32, 128], [0, 50, 60]),
    "32 heads on a key head": (32, 1, 400, 400, [0, 150, 400], [0, 150, 400]),
    "64 heads on a key head": (64, 1, 64, 64, [0, 22, 64], [0, 22, 64]),
    "128 heads on each key head": (256, 2, 9, 300, [0, 3, 5, 9], [0, 100, 210, 300]),
    "few rows of long keys": (5, 1, 6, 3001, [0, 1, 6], [0, 2990, 2993]),
    "few rows, the second document long": (3, 1, 10, 3001, [0, 6, 10], [0, 3, 3001]),
    "few rows, a key each": (5, 1, 6, 3001, [0, 1, 1, 6], [0, 1, 10, 11]),
    "one tile of long keys": (10, 2, 20, 3001, [0, 5, 20], [0, 2900, 2910]),
    "many short documents": (2, 1, 260, 200, [0, 30, 31, 90, 200, 260], [0, 5, 40, 70, 130, 200]),
}


@pytest.mark.parametrize("d,cap", [(64, 0.0), (128, 0.0), (64, 6.0)])
@pytest.mark.parametrize("causal,prefix", [(0, None), (16, None), (1, 30), (97, 7)])
@pytest.mark.parametrize("name", CASES)
def test_bias_by_distance_in_documents(name, causal, prefix, d, cap):
    import torch
    H, Hk, Nq, Nk, dq, dk = CASES[name]
    q, k, v = tensors(1, H, Hk, Nq, Nk, d, seed=40 + H)
    kw = dict(causal=causal, cap=cap, slopes=[0.01 * (1 + h % 7) for h in range(H)], docs_q=dq, docs_k=dk,
              prefix=None if prefix is None else [prefix] * (len(dq) - 1))
    check(*run(q, k, v, out_dtype=torch.float32, **kw), q, k, v, **kw)


def test_bias_that_grows_with_distance_in_documents():
    import torch
    q, k, v = tensors(2, 2, 2, 300, 100, 64, seed=50)
    kw = dict(slopes=[-0.05, 0.4], docs_q=[[0, 100, 300], [0, 290, 300]], docs_k=[[0, 40, 100], [0, 9, 100]])
    check(*run(q, k, v, out_dtype=torch.float32, **kw), q, k, v, **kw)
