"""GPU checks of the accumulated cache weights and the eviction against the 64-bit forms, and of one step of a
rolling cache (rotary positions, masked attention, weights, eviction) run together.

Weights tolerance: a score is off by e as in the masked forward's tests, lse in exp2 units by 2^-23 of itself, the
exponential by 2^-21; sums of n positive terms in short chains add 2^-18 (several hundred additions at most, each
2^-24): |w - want| <= (2 e + 2^-22 (|s| + |lse|) + 2^-17) sum + 2^-22 |decay w_in|."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from tests.test_gpu_masked import tensors

pytestmark = pytest.mark.gpu


def weights_want(q, k, lse, w, *, decay, causal=0, docs_q=None, docs_k=None, prefix=None, lengths=None, cap=0.0,
                 slopes=None, scale=None):
    B, H, Nq, d = q.shape
    Hk, Nk = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    q, k, lse = (x.double().cpu().numpy() for x in (q, k, lse))
    got = np.zeros((B, Hk, Nk))
    tol = np.zeros((B, Hk, Nk))
    row = lambda t, b: None if t is None else np.atleast_2d(t)[b % np.atleast_2d(t).shape[0]]  # noqa: E731
    for b in range(B):
        see, dist = O.visible(Nq, Nk, causal, row(docs_q, b), row(docs_k, b), row(prefix, b),
                              None if lengths is None else lengths[b])
        for h in range(H):
            hk = h // (H // Hk)
            sl = 0.0 if slopes is None else float(slopes[h])
            g = O.cache_weights(q[b, h], k[b, hk], lse[b, h], scale, see, cap=cap, slope=sl, dist=dist)
            kk = np.where(see.any(0)[:, None], k[b, hk], 0.0)
            live = np.isfinite(lse[b, h])
            a = abs(scale) * float((np.abs(np.where(live[:, None], q[b, h], 0)) @ np.abs(kk).T).max(initial=0.0))
            top = float(np.abs(lse[b, h][live]).max(initial=0.0))
            far = abs(sl) * float(dist.max(initial=0.0))
            e = d * 2.0 ** -23 * a + 2.0 ** -20 * cap + 2.0 ** -22 * far
            got[b, hk] += g
            tol[b, hk] += (2 * e + 2.0 ** -22 * (a + far + top) + 2.0 ** -17) * g
    if w is not None:
        w = w.double().cpu().numpy()
        got += decay * w
        tol += 2.0 ** -22 * np.abs(decay * w)
        if lengths is not None:
            for b, n in enumerate(lengths):
                got[b, :, max(n, 0):] = w[b, :, max(n, 0):]
                tol[b, :, max(n, 0):] = 0
    return got, tol


def case(H, Hk, Nq, Nk, d, seed=0, layout="bhnd", decay=0.9, **kw):
    from video_dit_sparse_gb300 import binding as sa
    B = len(kw["lengths"]) if kw.get("lengths") is not None else 2
    q, k, v = tensors(B, H, Hk, Nq, Nk, d, seed=seed, layout=layout)
    dev = {n: torch.tensor(x, dtype=torch.float32 if n == "slopes" else torch.int32, device="cuda")
           if n in ("docs_q", "docs_k", "prefix", "lengths", "slopes") and x is not None else x for n, x in kw.items()}
    _, lse = sa.sparse_attn_forward_masked(q, k, v, **dev)
    w = torch.rand(B, Hk, Nk, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sa.sparse_attn_cache_weights(q, k, lse, w, decay=decay, status=status, **dev)
    assert int(status) == 0
    want, tol = weights_want(q, k, lse, w, decay=decay, **kw)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(~(err <= tol))[:4])
    return q, k, v, lse, w, got, dev


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,Nq,Nk", [(1, 1, 1, 1), (2, 2, 1, 300), (3, 1, 2, 129), (8, 2, 70, 257), (2, 2, 300, 128),
                                        (6, 2, 259, 513), (1, 1, 1100, 90)])
@pytest.mark.parametrize("causal", [0, 1, 97])
def test_weights_sizes(d, H, Hk, Nq, Nk, causal):
    case(H, Hk, Nq, Nk, d, seed=Nq + Nk, causal=causal)


@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (6.0, True)])
@pytest.mark.parametrize("Nq", [1, 270])
def test_weights_cap_and_bias(cap, bias, Nq):
    case(4, 2, Nq, 333, 128, seed=5, layout="bnhd", cap=cap, causal=1,
         slopes=[0.5, 0.25, 0.125, 0.0625] if bias else None)


@pytest.mark.parametrize("causal,prefix", [(0, None), (1, None), (1, [30, 0, 5, 2]), (50, [0, 0, 0, 99])])
def test_weights_documents(causal, prefix):
    case(2, 1, 300, 400, 64, seed=6, causal=causal, docs_q=[0, 100, 100, 101, 290], docs_k=[0, 250, 260, 260, 390],
         prefix=prefix)


@pytest.mark.parametrize("Nq", [1, 150])
def test_weights_lengths_dead_rows_and_garbage(Nq):
    from video_dit_sparse_gb300 import binding as sa
    lengths = [0, 1, 128, 200, 300]
    q, k, v, lse, w, got, dev = case(4, 2, Nq, 300, 128, seed=7, lengths=lengths, causal=1)
    # what lies behind a sequence, and rows without a finite lse, must not matter
    for b, n in enumerate(lengths):
        k[b, :, n:] = float("nan")
    q = torch.where((lse == -float("inf"))[..., None], torch.full_like(q, float("nan")), q)
    assert torch.equal(sa.sparse_attn_cache_weights(q, k, lse, w, decay=0.9, **dev), got)
    # in place, and from nothing
    acc = w.clone()
    assert sa.sparse_attn_cache_weights(q, k, lse, acc, decay=0.9, out=acc, **dev) is acc
    assert torch.equal(acc, got)
    fresh = sa.sparse_attn_cache_weights(q, k, lse, **dev)
    want, tol = weights_want(torch.nan_to_num(q), torch.nan_to_num(k), lse, None, decay=0.0, lengths=lengths, causal=1)
    assert (np.abs(fresh.double().cpu().numpy() - want) <= tol).all()


def test_weights_are_the_columns_of_the_softmax():
    q, k, v, lse, w, got, _ = case(2, 2, 500, 700, 64, seed=8, decay=0.0)
    # every row's probabilities add up to one
    total = got.double().sum(-1)
    assert float((total - 500).abs().max()) <= 500 * 2.0 ** -14


def test_weights_repeat_and_stream():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v, lse, w, got, dev = case(4, 1, 999, 1000, 128, seed=9, causal=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = sa.sparse_attn_cache_weights(q, k, lse, w, decay=0.9, stream=s, **dev)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, got)


def test_weights_of_many_documents():
    """Units find their run of Q tiles among many; empty documents, rows of none, prefixes."""
    g = np.random.default_rng(3)
    nq, nk = g.integers(0, 120, 60), g.integers(0, 90, 60)
    docs_q, docs_k = ([int(x) for x in np.concatenate([[5], 5 + np.cumsum(n)])] for n in (nq, nk))
    case(2, 1, docs_q[-1] + 7, docs_k[-1] + 300, 64, seed=10, causal=9, docs_q=docs_q, docs_k=docs_k,
         prefix=[int(x) for x in g.integers(0, 40, 60)])


def test_results_made_on_another_stream():
    """What a call on a stream makes and fills is ordered with that stream, not with a busy current one."""
    from video_dit_sparse_gb300 import binding as sa
    q, k, v, lse, w, got, dev = case(2, 2, 40, 400, 64, seed=11, lengths=[400, 130, 0])
    docs = dict(docs_q=torch.tensor([0, 40], dtype=torch.int32, device="cuda"),
                docs_k=torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    want = sa.sparse_attn_cache_weights(q, k, lse, **dev)
    want_o, want_l = sa.sparse_attn_forward_masked(q, k, v, **docs)
    want_e = sa.sparse_attn_cache_evict(w, k, v, 200, sink=4, recent=8, lengths=dev["lengths"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    mine = sa.sparse_attn_cache_weights(q, k, lse, stream=s, **dev)
    o, l = sa.sparse_attn_forward_masked(q, k, v, stream=s, **docs)
    e = sa.sparse_attn_cache_evict(w, k, v, 200, sink=4, recent=8, lengths=dev["lengths"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(mine, want) and torch.equal(o, want_o) and torch.equal(l, want_l)
    assert all(torch.equal(a, b) for a, b in zip(e, want_e))


# ---------------------------------------------------------------- eviction

def evict_case(w, n_of, budget, sink, recent, d=64, layout="bhnd"):
    from video_dit_sparse_gb300 import binding as sa
    B, H, N = w.shape
    _, k, v = tensors(B, 1, H, 1, N, d, seed=1, layout=layout)
    lens = None if n_of is None else torch.tensor(n_of, dtype=torch.int32, device="cuda")
    out = (torch.full((B, H, budget, d), 5.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((B, budget, H, d), 6.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2),
           torch.full((B, H, budget), 7.0, device="cuda"))
    kept, ko, vo, wo = sa.sparse_attn_cache_evict(w.cuda(), k, v, budget, sink=sink, recent=recent, lengths=lens, out=out)
    for b in range(B):
        n = N if n_of is None else min(max(n_of[b], 0), N)
        for h in range(H):
            want = torch.from_numpy(O.evict(w[b, h].numpy(), n, budget, sink, recent)).cuda()
            m = len(want)
            assert torch.equal(kept[b, h, :m].long(), want), (b, h)
            assert bool((kept[b, h, m:] == -1).all())
            assert torch.equal(ko[b, h, :m], k[b, h, want]) and bool((ko[b, h, m:] == 5).all())
            assert torch.equal(vo[b, h, :m], v[b, h, want]) and bool((vo[b, h, m:] == 6).all())
            same = (wo[b, h, :m] == w[b, h].cuda()[want]) | torch.isnan(wo[b, h, :m])
            assert bool(same.all()) and bool((wo[b, h, m:] == 7).all())


@pytest.mark.parametrize("N,budget,sink,recent", [(1, 1, 0, 0), (2, 1, 1, 0), (33, 32, 0, 0), (1000, 1, 0, 0),
                                                  (1000, 999, 10, 20), (1025, 300, 0, 300), (4097, 2000, 1000, 1000),
                                                  (5000, 77, 7, 13), (60000, 30000, 100, 100)])
@pytest.mark.parametrize("kind", ["heavy", "ties", "equal"])
def test_evict(N, budget, sink, recent, kind):
    g = torch.Generator().manual_seed(N)
    w = torch.exp(3 * torch.randn(1, 3, N, generator=g))
    if kind == "ties":
        w = w.clamp(0.5, 2).mul(4).round() / 4
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    evict_case(w, None, budget, sink, recent)


def test_evict_lengths_and_layouts():
    w = torch.rand(6, 2, 500)
    evict_case(w, [0, 1, 99, 100, 101, 500], 100, 10, 20, d=128, layout="bnhd")
    evict_case(w, [-3, 10 ** 6, 3, 40, 41, 42], 40, 20, 20)
    evict_case(w, None, 700, 0, 0)  # a budget over the cache


def test_evict_signs_zeros_and_non_finite_weights():
    w = torch.randn(1, 2, 300)
    w[0, 0, ::3] = 0.0
    w[0, 0, 1::3] = -0.0
    w[0, 1, 5:50] = float("nan")
    w[0, 1, 60:90] = float("inf")
    w[0, 1, 90:120] = -float("inf")
    for budget in (10, 31, 150, 260, 299):
        evict_case(w, None, budget, 3, 4)


def test_evict_selects_only():
    from video_dit_sparse_gb300 import binding as sa
    w = torch.rand(2, 2, 200)
    kept, k, v, wo = sa.sparse_attn_cache_evict(w.cuda(), None, None, 50)
    assert k is None and v is None
    for b in range(2):
        for h in range(2):
            want = O.evict(w[b, h].numpy(), 200, 50, 0, 0)
            assert np.array_equal(kept[b, h].cpu().numpy(), want)
            assert torch.equal(wo[b, h].cpu(), w[b, h][want])


# ---------------------------------------------------------------- together

def test_one_step_of_a_rolling_cache():
    """Three chunks enter a cache that holds two and a half: rope, append, attend, accumulate, evict."""
    from video_dit_sparse_gb300 import binding as sa
    B, H, Hk, d, grid = 1, 4, 2, 64, (2, 6, 8)
    L, budget = 96, 240
    axes = (24, 20, 20)
    cap = 20.0
    kc = torch.zeros(B, Hk, budget + L, d, dtype=torch.bfloat16, device="cuda")
    vc, w = torch.zeros_like(kc), torch.zeros(B, Hk, budget + L, device="cuda")
    n = 0
    for step in range(4):
        g = torch.Generator().manual_seed(step)
        q, k, v = (torch.randn(B, L, h, d, generator=g).to(torch.bfloat16).cuda().transpose(1, 2) for h in (H, Hk, Hk))
        slot = slice(n, n + L)
        qr, _ = sa.sparse_attn_rope(q, k, axes=axes, grid=grid, offset=(2 * step, 0, 0), out=(None, kc[:, :, slot]))
        want = O.rope(q.double().cpu().numpy(), O.voxel_positions(grid, None, (2 * step, 0, 0)), axes)
        assert np.abs(qr.double().cpu().numpy() - want).max() <= 2.0 ** -8 * 8
        vc[:, :, slot] = v
        w[:, :, slot] = 0
        n += L
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        o, lse = sa.sparse_attn_forward_masked(qr, kc, vc, cap=cap, causal=48, lengths=lens)
        from tests.test_gpu_masked import check
        check(o, lse, qr, kc, vc, cap=cap, causal=48, lengths=[n])
        before = w.clone()
        sa.sparse_attn_cache_weights(qr, kc, lse, w, decay=0.5, cap=cap, causal=48, lengths=lens, out=w)
        got, tol = weights_want(qr, kc, lse, before, decay=0.5, cap=cap, causal=48, lengths=[n])
        assert (np.abs(w.double().cpu().numpy() - got) <= tol).all()
        if n > budget:
            kept, k2, v2, w2 = sa.sparse_attn_cache_evict(w, kc, vc, budget, sink=48, recent=48, lengths=lens)
            for h in range(Hk):
                idx = O.evict(w[0, h].cpu().numpy(), n, budget, 48, 48)
                assert np.array_equal(kept[0, h].cpu().numpy(), idx)
                assert torch.equal(k2[0, h], kc[0, h, torch.from_numpy(idx).cuda()])
            kc[:, :, :budget], vc[:, :, :budget], w[:, :, :budget] = k2, v2, w2
            n = budget
    assert n == budget


@pytest.mark.parametrize("causal,cap", [(0, 0.0), (33, 0.0), (1, 9.0), (0, 9.0)])
@pytest.mark.parametrize("H,Hk,Nq,Nk", [(1, 1, 3000, 70), (4, 2, 1500, 300), (84, 84, 40, 600), (128, 1, 9, 200)])
def test_weights_shared_and_many_units(H, Hk, Nq, Nk, causal, cap):
    """Few keys: a cluster shares a unit's rows.  Many units: a block takes several."""
    q, k, v, lse, w, got, dev = case(H, Hk, Nq, Nk, 64, seed=31, causal=causal, cap=cap)
    from video_dit_sparse_gb300 import binding as sa
    acc = w.clone()
    sa.sparse_attn_cache_weights(q, k, lse, acc, decay=0.9, out=acc, **dev)
    assert torch.equal(acc, got)


def test_weights_large_scores_under_a_cap():
    """Scores past the polynomial's range: the tile is summed again exactly."""
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(1, 2, 2, 300, 400, 64, seed=32, sigma=6.0)
    k[:, :, 200:] = float("inf")  # behind the sequence
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    _, lse = sa.sparse_attn_forward_masked(q, k, torch.nan_to_num(v), cap=7.0, lengths=lens)
    got = sa.sparse_attn_cache_weights(q, k, lse, cap=7.0, lengths=lens)
    want, tol = weights_want(q, torch.nan_to_num(k, posinf=0.0), lse, None, decay=0.0, cap=7.0, lengths=[200])
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("B,H,N,budget", [(1, 1, 500000, 1000), (77, 1, 50000, 49000), (1, 2, 8193, 8192), (2, 3, 40000, 20),
                                          (5, 9, 9000, 4000), (1, 2, 200001, 100000), (32, 5, 8500, 77)])
def test_evict_long_rows(B, H, N, budget):
    from video_dit_sparse_gb300 import binding as sa
    g = torch.Generator(device="cuda").manual_seed(N)
    w = torch.rand(B, H, N, generator=g, device="cuda").mul(1 << 12).round() / (1 << 12)  # many ties
    kept, _, _, wo = sa.sparse_attn_cache_evict(w, None, None, budget, sink=3, recent=5)
    assert torch.equal(wo, w.gather(2, kept.long()))
    for b, h in ((0, 0), (B - 1, H - 1)):
        want = O.evict(w[b, h].cpu().numpy(), N, budget, 3, 5)
        assert np.array_equal(kept[b, h].cpu().numpy(), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sink,recent", [(0, 0), (130, 200), (128, 0), (0, 128), (389, 388), (777, 0), (0, 777), (65, 711)])
def test_evict_rows_that_need_no_choice(d, sink, recent):
    """Tiles of only first or newest entries move before the others are chosen; tiles that hold both do not."""
    w = torch.rand(6, 2, 1500, generator=torch.Generator().manual_seed(sink + recent))
    evict_case(w, [1500, 777, 778, 900, 10, 0], 777, sink, recent, d=d, layout="bnhd")
    evict_case(w, None, 777, sink, recent, d=d)


def test_a_step_in_a_graph():
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(1, 4, 2, 1, 2000, 64, seed=33)
    lens = torch.tensor([1500], dtype=torch.int32, device="cuda")
    w = torch.rand(1, 2, 2000, device="cuda")
    kept = torch.empty(1, 2, 700, dtype=torch.int32, device="cuda")
    out = (torch.zeros(1, 2, 700, 64, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(1, 2, 700, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 700, device="cuda"))

    def step():
        o, lse = sa.sparse_attn_forward_masked(q, k, v, lengths=lens)
        acc = sa.sparse_attn_cache_weights(q, k, lse, w, lengths=lens)
        sa.sparse_attn_cache_evict(acc, k, v, 700, recent=10, lengths=lens, out=out, kept=kept)
        return o, acc
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, acc = step()
    for n in (1999, 3, 800):
        lens.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, acc, kept)]
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], kept)


@pytest.mark.parametrize("H,Hk,Nq,Nk,causal,key", [(1, 1, 1, 300, 0, 5), (3, 1, 200, 200, 1, 190), (3, 1, 200, 500, 1, 490),
                                                  (6, 2, 100, 300, 33, 299), (2, 2, 40, 300, 0, 7)])
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_weights_of_a_key_that_is_not_finite(H, Hk, Nq, Nk, causal, key, cap):
    """Rows whose score is -inf give the key nothing; rows without a finite lse add nothing to any key; rows that do not
    see it do not meet it.  So a key with such a score keeps decay * w."""
    from video_dit_sparse_gb300 import binding as sa
    q, k, v = tensors(1, H, Hk, Nq, Nk, 64, seed=41)
    w = torch.rand(1, Hk, Nk, device="cuda")
    k0 = k.clone()
    k0[:, :, key] = 0
    for bad in ("nan", "low") if cap == 0 else ("nan",):  # (under a cap the score of -inf is -cap)
        if bad == "nan":
            k[:, :, key] = float("nan")
        else:
            q[..., 9] = q[..., 9].abs() + 0.25
            k[:, :, key] = 0
            k[:, :, key, 9] = -float("inf")
        _, lse = sa.sparse_attn_forward_masked(q, k, v, causal=causal, cap=cap)
        got = sa.sparse_attn_cache_weights(q, k, lse, w, decay=0.9, causal=causal, cap=cap)
        want, tol = weights_want(q, k0, lse, None, decay=0.0, causal=causal, cap=cap)
        want[:, :, key] = tol[:, :, key] = 0
        w64 = w.double().cpu().numpy()
        want, tol = want + 0.9 * w64, tol + 2.0 ** -22 * np.abs(0.9 * w64)
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
