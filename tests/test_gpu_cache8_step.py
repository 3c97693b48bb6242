"""A run of the operators as a rolling cache uses them: rows normalised and rotated, keys and values into the 8-bit cache,
attention over it; in one captured step, replayed with other tokens and lengths.

Tolerances: the attention's are those of test_gpu_attend8.py, on the values that the cache holds."""
import pytest
import torch

from tests.test_gpu_attend8 import check

pytestmark = pytest.mark.gpu


def test_generation_steps_in_one_graph():
    from video_dit_sparse_gb300 import binding as sa
    B, H, Hk, d, room = 2, 8, 2, 128, 400
    g = torch.Generator().manual_seed(1)
    qkv = torch.zeros(B, 1, H + 2 * Hk, d, dtype=torch.bfloat16, device="cuda")  # a fused projection's output
    q, k, v = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
    w = [(1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    lengths, pos = at + 1, at.view(B, 1, 1).clone()
    c = sa.sparse_attn_cache8(B, Hk, room, d, block=64)

    def step():
        qr, kr = sa.sparse_attn_norm_rope(q, k, q_weight=w[0], k_weight=w[1], axes=(128,), pairing="half", positions=pos)
        sa.sparse_attn_cache8_append(c, kr, v, at)
        return qr, kr, *sa.sparse_attn_forward_cache8(qr, c, causal=1, lengths=lengths)
    step()
    for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, kr, o, lse = step()
    first = torch.tensor([0, 131], dtype=torch.int32)  # the second sequence has a prompt
    prompt = torch.randn(B, Hk, 131, d, generator=g).to(torch.bfloat16).cuda()
    sa.sparse_attn_cache8_append(c, prompt, prompt, 0, counts=torch.tensor([0, 131], dtype=torch.int32, device="cuda"))
    keys = [[], []]
    for n in range(70):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        at.copy_(first + n)
        lengths.copy_(first + n + 1)
        pos.copy_((first + n).view(B, 1, 1))
        graph.replay()
        for b in range(B):
            keys[b].append(kr[b].clone())
        if n in (0, 1, 63, 64, 69):
            check(o, lse, qr, c, causal=1, lengths=lengths.tolist())
    # what the cache holds are the keys that went in: each code within half a step, at the scale of its own time or a
    # larger one: twice 2^-4 of the value and 2^-9 of the final scale at most
    got, _ = sa.sparse_attn_cache8_read(c, first.cuda(), 70, out_dtype=torch.float32)
    per = c.k_scale.repeat_interleave(64, -1)
    for b in range(B):
        want = torch.cat(keys[b], 1).float()
        s = per[b][:, first[b]:first[b] + 70, None]
        assert bool(((got[b] - want).abs() <= want.abs() * 2.0 ** -3 + s * 2.0 ** -9).all())


def test_a_chunk_over_the_window_against_the_bf16_path():
    """The cache read back and attended by the bf16 kernel gives the same rows: both round weights to ten bits or eight."""
    from video_dit_sparse_gb300 import binding as sa
    B, H, d, frame, room = 1, 3, 128, 60, 600
    g = torch.Generator().manual_seed(2)
    make = lambda n: torch.randn(B, n, H, d, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)  # noqa: E731
    c = sa.sparse_attn_cache8(B, H, room, d, block=32)
    for n in range(0, room, 240):
        x, y, z = make(min(240, room - n)), make(min(240, room - n)), make(min(240, room - n))
        grid = dict(grid=(x.shape[2] // frame, 6, 10), offset=(n // frame, 0, 0))
        qr, kr = sa.sparse_attn_norm_rope(x, y, norm="layer", **grid)
        sa.sparse_attn_cache8_append(c, kr, z, n)
        lengths = torch.tensor([n + x.shape[2]], dtype=torch.int32, device="cuda")
        o, lse = sa.sparse_attn_forward_cache8(qr, c, causal=frame, lengths=lengths, out_dtype=torch.float32)
        k, v = sa.sparse_attn_cache8_read(c, 0, room)
        o2, lse2 = sa.sparse_attn_forward_masked(qr, k, v, causal=frame, lengths=lengths, out_dtype=torch.float32)
        # weights: 2^-8 (bf16) and 2^-10 of each, so of o at most that times sum p |v| / 1 <= max |v|
        assert float((o - o2).abs().max()) <= (2.0 ** -8 + 2.0 ** -10) * 1.1 * 2 * float(v.float().abs().max())
        # scores: bf16 products exact, the row's two terms off by 2^-17 of its largest value
        e = 2.0 ** -17 * d ** -0.5 * float(qr.abs().max()) * float(k.abs().sum(-1).max()) + 2.0 ** -16 * 20
        assert float((lse - lse2).abs().max()) <= e
        check(o, lse, qr, c, causal=frame, lengths=lengths.tolist())


def test_training_step_gradients():
    """A layer that learns its norms: the gradient of a loss of the rotated rows, by the library and by differences."""
    from video_dit_sparse_gb300 import binding as sa
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 4, 33, 64, generator=g).cuda()
    w, b = (1 + 0.2 * torch.randn(64, generator=g)).cuda(), (0.2 * torch.randn(64, generator=g)).cuda()
    target = torch.randn(2, 4, 33, 64, generator=g).cuda()
    opt = dict(norm="layer", axes=(16, 24, 24), grid=(3, 11, 1))

    def loss(w, b):
        y = sa.sparse_attn_norm_rope(x, q_weight=w, q_bias=b, **opt)
        return 0.5 * ((y - target).double() ** 2).sum(), y - target
    _, dy = loss(w, b)
    dx, dw, db = sa.sparse_attn_norm_rope_backward(dy, None, x, q_weight=w, q_bias=b, **opt)
    for i in (0, 17, 63):
        for vec, grad in ((w, dw), (b, db)):
            up, down = vec.clone(), vec.clone()
            up[i] += 2.0 ** -5
            down[i] -= 2.0 ** -5
            pair = [loss(*((t, b) if vec is w else (w, t)))[0] for t in (up, down)]
            # the loss is quadratic in both vectors, so the difference is exact but for fp32: 264 rows of terms of a few
            # units, each within 2^-18, over the step
            assert abs(float((pair[0] - pair[1]) / 2.0 ** -4) - float(grad[i])) <= 264 * 64 * 2.0 ** -18 * 8 / 2.0 ** -4 / 16
