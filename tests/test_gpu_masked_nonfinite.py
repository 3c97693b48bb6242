"""GPU checks of what keys and values that a row does not see may hold: anything.  Of what it sees, a value that is not
finite comes out, and a score that is not a number makes the row's output and lse none.

A row is compared with the 64-bit form on the same inputs with the poisoned keys and values replaced by zeros (rows that
do not see them cannot tell the difference), within test_gpu_masked's tolerances."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from tests.test_gpu_masked import check, run, tensors

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def sees_any(B, H, Nq, Nk, poisoned, causal=0, docs_q=None, docs_k=None, prefix=None, lengths=None, **_):
    """bool [B, H, Nq]: the row sees a poisoned key."""
    out = np.zeros((B, H, Nq), dtype=bool)
    for b in range(B):
        see, _ = O.visible(Nq, Nk, causal, docs_q, docs_k, prefix, None if lengths is None else lengths[b])
        out[b] = see[:, poisoned].any(1)
    return out


def poisoned_case(H, Hk, Nq, Nk, d, poisoned, bad, *, with_k, out_dtype=torch.float32, B=1, seed=60, in_place=False, **kw):
    q, k, v = tensors(B, H, Hk, Nq, Nk, d, seed=seed)
    if with_k:
        k[:, :, poisoned] = bad
    v[:, :, poisoned] = bad
    k0, v0 = k.clone(), v.clone()
    k0[:, :, poisoned] = 0
    v0[:, :, poisoned] = 0
    clean_o, clean_l = run(q, k0, v0, out_dtype=out_dtype, **kw)
    q_in = q.clone()
    o, lse = run(q_in, k, v, out_dtype=out_dtype, out=q_in if in_place else None, **kw)
    hit = torch.from_numpy(sees_any(B, H, Nq, Nk, poisoned, **kw)).cuda()
    assert bool(hit.any()) or not bool(hit.numel())
    # (rows that see the poison stand aside: the clean run's take their place in the comparison)
    check(torch.where(hit[..., None], clean_o, o), torch.where(hit, clean_l, lse), q, k0, v0, **kw)
    if not with_k:
        assert bool((~torch.isfinite(o[hit])).all())
        assert torch.equal(lse[hit], run(q, k, v0, out_dtype=out_dtype, **kw)[1][hit])
    else:
        assert bool(torch.isnan(o[hit]).all())
        if np.isnan(bad):
            assert bool(torch.isnan(lse[hit]).all())


PACKED = {  # H, Hk, Nq, Nk, tables, poisoned keys (one document's, or a part of it)
    "second of two in one unit": (1, 1, 256, 512, dict(docs_q=[0, 128, 256], docs_k=[0, 100, 512]), slice(100, 512)),
    "first of two in one unit": (1, 1, 256, 512, dict(docs_q=[0, 128, 256], docs_k=[0, 100, 512]), slice(0, 100)),
    "inside a tile of rows": (2, 1, 200, 300, dict(docs_q=[0, 37, 41, 200], docs_k=[0, 60, 150, 300]), slice(60, 150)),
    "one key of the next document": (2, 2, 100, 200, dict(docs_q=[0, 50, 100], docs_k=[0, 90, 200]), slice(90, 91)),
    "shared heads, frames": (8, 2, 150, 300, dict(docs_q=[0, 70, 150], docs_k=[0, 140, 300], causal=16), slice(140, 300)),
    "prefix": (1, 1, 260, 260, dict(docs_q=[0, 130, 260], docs_k=[0, 130, 260], causal=1, prefix=[20, 9]), slice(0, 130)),
    "few rows, split keys": (3, 1, 9, 9001, dict(docs_q=[0, 2, 9], docs_k=[0, 7000, 9000]), slice(0, 7000)),
    "one tile, split keys": (10, 2, 20, 3001, dict(docs_q=[0, 5, 20], docs_k=[0, 1900, 3001]), slice(1900, 3001)),
    "later keys of the causal rows": (2, 1, 400, 400, dict(causal=1), slice(203, 204)),
    "a later frame": (12, 3, 64, 1000, dict(causal=32), slice(980, 1000)),
    "a few causal rows": (1, 1, 7, 4000, dict(causal=1), slice(3996, 4000)),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad,with_k", [(NAN, True), (NAN, False), (INF, False), (-INF, False)])
@pytest.mark.parametrize("name", PACKED)
def test_rows_that_do_not_see_them(name, bad, with_k, d):
    H, Hk, Nq, Nk, kw, poisoned = PACKED[name]
    poisoned_case(H, Hk, Nq, Nk, d, poisoned, bad, with_k=with_k, **kw)


@pytest.mark.parametrize("kw", [dict(cap=9.0), dict(slopes=[0.05, 0.2]), dict(cap=9.0, slopes=[0.05, -0.01])])
@pytest.mark.parametrize("name", ["inside a tile of rows", "later keys of the causal rows"])
def test_rows_that_do_not_see_them_with_a_cap_and_a_bias(name, kw):
    H, Hk, Nq, Nk, tables, poisoned = PACKED[name]
    poisoned_case(H, Hk, Nq, Nk, 128, poisoned, NAN, with_k=False, **tables, **kw)


@pytest.mark.parametrize("name", ["second of two in one unit", "later keys of the causal rows", "few rows, split keys"])
def test_in_place_and_bf16(name):
    H, Hk, Nq, Nk, kw, poisoned = PACKED[name]
    poisoned_case(H, Hk, Nq, Nk, 128, poisoned, NAN, with_k=False, in_place=True, out_dtype=torch.bfloat16, **kw)


def test_more_units_than_blocks():
    """Blocks go on to the next unit after rows that were computed again."""
    n = 900
    poisoned_case(42, 42, n, n, 64, slice(450, 700), NAN, B=2, with_k=False, causal=1, docs_q=[0, 449, n], docs_k=[0, 451, n])


def test_each_column_on_its_own():
    """A value that is not finite reaches its own column of the rows that see it, and no other."""
    q, k, v = tensors(1, 2, 1, 300, 300, 128, seed=61)
    v[0, 0, 200, 5], v[0, 0, 210, 100], v[0, 0, 220, 64] = NAN, INF, -INF
    v0 = torch.nan_to_num(v, posinf=0.0, neginf=0.0)
    o, lse = run(q, k, v, causal=1, out_dtype=torch.float32)
    want, wl = run(q, k, v0, causal=1, out_dtype=torch.float32)
    assert torch.equal(lse, wl)
    for column, key, bad in ((5, 200, NAN), (100, 210, INF), (64, 220, -INF)):
        seen = o[0, :, key:, column]
        assert bool(torch.isnan(seen).all()) if np.isnan(bad) else bool((seen == bad).all())
        o[0, :, key:, column] = want[0, :, key:, column]
    check(o, lse, q, k, v0, causal=1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,Nk", [(4, 2, 1, 9001), (1, 1, 1, 880), (3, 1, 10, 3001), (40, 1, 2, 3001), (2, 2, 300, 700)])
def test_an_infinite_value_that_every_row_sees(H, Hk, Nq, Nk, d):
    """It comes out as it is, in its own column: split keys and rows in every lane quarter included."""
    q, k, v = tensors(1, H, Hk, Nq, Nk, d, seed=63, sigma=0.5)
    v[0, 0, Nk // 2, 7], v[0, 0, 100, 9], v[0, 0, Nk - 2, 20] = INF, -INF, NAN
    v0 = torch.nan_to_num(v, posinf=0.0, neginf=0.0)
    o, lse = run(q, k, v, out_dtype=torch.float32)
    want, wl = run(q, k, v0, out_dtype=torch.float32)
    assert torch.equal(lse, wl)
    heads = slice(0, H // Hk)
    assert bool((o[0, heads, :, 7] == INF).all()) and bool((o[0, heads, :, 9] == -INF).all())
    assert bool(torch.isnan(o[0, heads, :, 20]).all())
    for column in (7, 9, 20):
        o[0, heads, :, column] = want[0, heads, :, column]
    check(o, lse, q, k, v0)
