"""The 64-bit formulas of tests/blocks64.py: each gradient against central
differences of its own forward, and the routing against hand-made rows."""
from __future__ import annotations

import pytest
import torch

from tests import blocks64 as B

F64 = torch.float64
# central differences of step h: error h^2 f''' / 6 + 2^-52 |f| / h, about 1e-9 at h = 1e-5 for
# functions and derivatives of order 1 .. 100
STEP, TOL = 1e-5, 2e-7


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64)


def _slope(f, x, v):
    return (f(x + STEP * v) - f(x - STEP * v)) / (2 * STEP)


def _close(a, b):
    assert abs(a - b) <= TOL * max(1.0, abs(a), abs(b)), (float(a), float(b))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference_quotient(kind, renorm):
    gen = torch.Generator().manual_seed(1)
    x = _randn(gen, 5, 13)
    x[1, 3] = -B.INF
    ids, _ = B.route(x, 4, kind, renorm=renorm)
    ids[2, 3] = -1
    dw = _randn(gen, 5, 4)
    dx = B.route_backward(x, ids, dw, kind, renorm, 1.7)
    for _ in range(6):
        v = _randn(gen, 5, 13)
        _close(_slope(lambda z: (B.route_weights(z, ids, kind, renorm, 1.7) * dw).sum(), x, v),
               (dx * v).sum())


def test_swiglu_gradient_is_the_difference_quotient():
    gen = torch.Generator().manual_seed(2)
    x, dy, w = _randn(gen, 3, 16), _randn(gen, 3, 8), _randn(gen, 3).abs()
    dx, dw = B.swiglu_backward(x, dy, w)
    v, vw = _randn(gen, 3, 16), _randn(gen, 3)
    _close(_slope(lambda z: (B.swiglu(z, w) * dy).sum(), x, v), (dx * v).sum())
    _close(_slope(lambda z: (B.swiglu(x, z) * dy).sum(), w, vw), (dw * vw).sum())


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients_are_the_difference_quotients(post, gated, weighted):
    gen = torch.Generator().manual_seed(3)
    T, C, a = 4, 24, 0.6
    r, h, dr, dx = (_randn(gen, T, C) for _ in range(4))
    gate = _randn(gen, T, C) if gated else None
    wp, wq = (_randn(gen, C), _randn(gen, C)) if weighted else (None, None)

    def loss(r=r, h=h, gate=gate, wp=wp, wq=wq):
        r1, x, _, _ = B.residual_norm(r, h, wp, gate, wq, post, a)
        return (r1 * dr).sum() + (x * dx).sum()

    r1, _, p, q = B.residual_norm(r, h, wp, gate, wq, post, a)
    d = B.residual_norm_backward(dr, r1, h, dx, wp, gate, wq, p, q, a)
    for name, x, g in (("r", r, d[0]), ("h", h, d[1]), ("gate", gate, d[2]), ("wp", wp, d[3]),
                       ("wq", wq, d[4])):
        if x is not None:
            v = _randn(gen, *x.shape)
            _close(_slope(lambda z: loss(**{name: z}), x, v), (g * v).sum())


def test_route_by_hand():
    inf = B.INF
    x = torch.tensor([[1.0, 3.0, 3.0, -inf, 2.0, 0.0], [-inf] * 6, [float("nan"), inf, 1.0, 0, 0, 0],
                      [-inf, -inf, 5.0, -inf, -inf, 1.0]], dtype=F64)
    ids, w = B.route(x, 3, "softmax")
    # ties to the lowest index; no expert at all; +inf counts as the largest number and takes all
    assert ids.tolist() == [[1, 2, 4], [-1, -1, -1], [1, 2, 3], [2, 5, -1]]
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [1, 0, 0]
    assert abs(float(w[3].sum()) - 1) < 1e-15 and float(w[3, 2]) == 0
    # two of three groups of two by their best two keys: sums 4, 3 (of one expert), 2
    ids, _ = B.route(torch.tensor([[1.0, 3.0, 3.0, -inf, 2.0, 0.0]], dtype=F64), 4, "sigmoid",
                     groups=3, topk_groups=2)
    s = torch.sigmoid(torch.tensor([1.0, 3.0, 2.0, 0.0], dtype=F64))
    assert s[0] + s[1] > s[2] + s[3] > s[1]          # groups 0 and 2 win
    assert ids.tolist() == [[1, 4, 0, 5]]
    # a bias moves the choice and no weight
    bias = torch.tensor([0, 0, 0, 0, 9.0, -inf], dtype=F64)
    ids, w = B.route(torch.zeros(1, 6, dtype=F64), 6, "softmax", bias=bias, renorm=False)
    assert ids.tolist() == [[4, 0, 1, 2, 3, -1]]
    assert torch.allclose(w[0, :5], torch.full((5,), 1 / 6, dtype=F64))
