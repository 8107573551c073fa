"""GPU tests of the rotary calls at their limits: angles of far positions from frequencies to the last
unit, and gradients."""
import decimal
import math

import numpy as np
import pytest
import torch

from test_gpu_rope import F32, f64, i32, rand, sv  # noqa: F401

pytestmark = pytest.mark.gpu

TAU = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257242")


@pytest.mark.parametrize("at", [1, 131071, 2 ** 31 - 2, -70000, -2 ** 31])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions_to_the_bound(sv, at, base):  # noqa: F811
    """At any position a component is off by no more than 2^-21 of its pair's length: a frequency's
    half unit of 2^-64 of a turn is 2^-31 radians at most."""
    rot = 64
    with decimal.localcontext() as c:
        c.prec = 70
        turns = [(-(decimal.Decimal(2 * i) / rot) * decimal.Decimal(base).ln()).exp() / TAU
                 for i in range(rot // 2)]
        angle = np.array([[2 * math.pi * float(p * x % 1) for x in turns] for p in (at, at + 1)])
    x = rand((1, 2, 3, rot), 1, F32)
    xs, c, s = f64(x), np.cos(angle)[None, :, None], np.sin(angle)[None, :, None]
    a, b = xs[..., :rot // 2], xs[..., rot // 2:]
    want, size = np.concatenate([a * c - b * s, b * c + a * s], -1), np.hypot(a, b)
    size = np.concatenate([size, size], -1)
    rope = sv.Rope(rot, base=base)
    for kw in (dict(pos=i32([[at, at + 1]])), dict(start=i32([at]))):
        got = f64(sv.sv_rope(rope, x, **kw))
        assert (np.abs(got - want) <= size * 2.0 ** -21 + np.abs(want) * 2.0 ** -24 * 1.001).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F32])
@pytest.mark.parametrize("how", ["start", "pos", "tree", "ragged"])
def test_graph_of_gradients(sv, dtype, how):  # noqa: F811
    """A tensor that requires grad keeps its graph: the gradient is the inverse rotation's, bit for
    bit, for dense and broadcast gradients, slices and tokens that are not there."""
    rope = sv.Rope(40, gain=1.5, interleaved=True)
    B, T, H, D = 2, 9, 3, 80
    kw = dict(start=i32([3, 7000]))
    if how == "pos":
        kw = dict(pos=i32([[5 * t + b for t in range(T)] for b in range(B)]))
    if how == "tree":
        kw["parent"] = i32([[0, 0, 0, 1, 1, 2, 4, 4, 7]] * B)
    if how == "ragged":
        kw["n_new"] = i32([T, 4])
    wide = rand((B, T, H + 2, D), 5, dtype).requires_grad_()
    g = rand((B, T, H, D), 6, dtype)
    y = sv.sv_rope(rope, wide[:, :, 1:-1], **kw)
    with torch.no_grad():
        plain = sv.sv_rope(rope, wide[:, :, 1:-1], **kw)
    assert torch.equal(y, plain) and y.requires_grad and not plain.requires_grad
    back = sv.sv_rope(rope, g, inverse=True, **kw)
    (got,) = torch.autograd.grad(y, wide, g, retain_graph=True)
    assert torch.equal(got[:, :, 1:-1], back) and not got[:, :, [0, -1]].any()
    if how == "ragged":
        assert not got[1, 4:].any()
    # (The gradient of a sum is one number, broadcast.)
    (got,) = torch.autograd.grad(y.sum(), wide)
    assert torch.equal(got[:, :, 1:-1], sv.sv_rope(rope, torch.ones_like(g), inverse=True, **kw))
    # A row that all share.
    row = rand((1, T, H, D), 7, dtype).requires_grad_()
    (got,) = torch.autograd.grad(sv.sv_rope(rope, row.expand(B, -1, -1, -1), **kw), row, g)
    assert torch.equal(got, back.sum(0, keepdim=True))
    assert rope.status() == sv.SV_OK


def test_gradients_against_differences(sv):  # noqa: F811
    """And against the map itself, which is linear: the sum over x of a step times the gradient is
    the sum over out of the difference times g. Components of x, of the step and of g are off by
    2^-21 of 1.5 times lengths below 12."""
    rope = sv.Rope(80, gain=1.5)
    x, g = rand((2, 9, 1, 80), 5, F32).requires_grad_(), rand((2, 9, 1, 80), 6, F32)
    kw = dict(start=i32([3, 7000]))
    (dx,) = torch.autograd.grad(sv.sv_rope(rope, x, **kw), x, g, create_graph=True)
    rng = np.random.default_rng(0)
    with torch.no_grad():
        y = f64(sv.sv_rope(rope, x, **kw))
        for _ in range(8):
            e = rand(x.shape, 10 + int(rng.integers(100)), F32)
            d = f64(sv.sv_rope(rope, x + e, **kw)) - y
            moved = f64(x + e) - f64(x)
            bound = 2.0 ** -21 * 1.5 * 12 * 3 * np.abs(f64(g)).sum()
            assert abs((d * f64(g)).sum() - (moved * f64(dx)).sum()) <= bound


def test_gradients_of_gradients_and_inverse(sv):  # noqa: F811
    rope = sv.Rope(64)
    x, g = (rand((1, 5, 2, 64), s, F32).requires_grad_() for s in (1, 2))
    (dx,) = torch.autograd.grad(sv.sv_rope(rope, x, inverse=True), x, g, create_graph=True)
    assert torch.equal(dx, sv.sv_rope(rope, g.detach()))
    (dg,) = torch.autograd.grad(dx, g, x.detach())
    assert torch.equal(dg, sv.sv_rope(rope, x.detach(), inverse=True))


def test_gradients_in_a_cuda_graph(sv):  # noqa: F811
    """Forward and backward captured, replayed on new values."""
    rope = sv.Rope(64)
    x, g = rand((2, 7, 3, 64), 1, F32).requires_grad_(), rand((2, 7, 3, 64), 2, F32)
    start = i32([4, 90])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.autograd.grad(sv.sv_rope(rope, x, start=start), x, g)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sv.sv_rope(rope, x, start=start)
        (dx,) = torch.autograd.grad(y, x, g)
    for seed in (3, 4):
        with torch.no_grad():
            x.copy_(rand(x.shape, seed, F32))
        g.copy_(rand(x.shape, seed + 10, F32))
        start.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, sv.sv_rope(rope, x.detach(), start=start))
        assert torch.equal(dx, sv.sv_rope(rope, g, start=start, inverse=True))


def test_gradients_with_a_stream(sv):  # noqa: F811
    rope, x = sv.Rope(64), rand((1, 5, 2, 64), 1, F32).requires_grad_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = sv.sv_rope(rope, x, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    (dx,) = torch.autograd.grad(y, x, torch.ones_like(y))
    assert torch.equal(y, sv.sv_rope(rope, x.detach()))
    assert torch.equal(dx, sv.sv_rope(rope, torch.ones_like(y), inverse=True))
