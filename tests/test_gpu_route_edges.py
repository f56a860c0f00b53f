"""Routing where the chosen experts' scores are tiny, against the 64-bit formulas.

A bias, or ids given by the caller, can choose experts whose scores lie far below the smallest binary32
number, while the renormalised weights, ratios of them, are of order one.

Error bounds, u = 2^-24: a ratio is made of exponentials of differences of logits, each rounded once
(|difference| u) and 2 ulp off, and then of the same sums, products and divisions as anywhere else, so
the bounds of test_gpu_route hold with `spread` the largest difference of two logits of a row, here
without a cap: (2 spread + 64) u of a weight, (2 spread + 96) u of the magnitudes of a gradient's terms."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import blocks64 as B
from tests.test_gpu_route import _grad_bound

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


def _spread(x):
    x = torch.where(x > -INF, x.double(), NAN)
    return (x.nan_to_num(-INF).amax(1) - x.nan_to_num(INF).amin(1)).clamp(min=0)[:, None]


# how far the chosen logits lie below 0 and below the row's largest logit: scores that are ordinary,
# subnormal, and no binary32 number at all
DEPTHS = [20.0, 87.0, 95.0, 101.0, 140.0, 300.0, 600.0]


def _low(T, E, seed, dtype):
    """Rows whose first quarter of experts is near 0 and the rest near -depth (kind softmax), or all
    near -depth from column E // 4 on; the depth changes from row to row."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=gen)
    depth = torch.tensor([DEPTHS[t % len(DEPTHS)] for t in range(T)])[:, None]
    x[:, E // 4:] -= depth
    return x.to(dtype), gen


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(24, 5), (256, 8), (1000, 32)])
def test_gradient_of_tiny_scores(cuda_device, dtype, kind, E, k):
    T = 29
    x, gen = _low(T, E, E + k, dtype)
    ids = torch.stack([torch.randperm(E - E // 4, generator=gen)[:k] + E // 4 for _ in range(T)]).int()
    ids[::5, 1] = -1
    dw = torch.randn(T, k, generator=gen) * 5
    for renorm in (True, False):
        ref = B.route_backward(x.double(), ids, dw.double(), kind, renorm, 1.5)
        got = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device), dw.to(cuda_device),
                                      scores=kind, renormalize=renorm, scale=1.5).cpu().double()
        bound = (2 * _spread(x) + 96) * U * _grad_bound(x.double(), ids, dw.double(), kind, renorm, 1.5)
        if dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * ref.abs()
        assert torch.isfinite(got).all()
        # a non-renormalised gradient may underflow: the smallest normal number times what it is multiplied by
        assert (got - ref).abs().le(bound + 2.0 ** -120).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_given_by_hand(cuda_device, kind):
    x = torch.tensor([[100.0, 5.0, 4.0, 3.0], [0.0, -90.0, -91.0, -92.0]])
    ids = torch.tensor([[1, 2], [1, 2]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -1.0], [100.0, -100.0]])
    got = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device), dw.to(cuda_device), scores=kind)
    # weights 1 / (1 + e^-1) and its complement: slope w (1 - w) of their difference, twice; the first
    # row's sigmoids are ordinary
    slope = 2 * 0.7310585786300049 * 0.2689414213699951
    want = torch.tensor([[0, slope, -slope, 0], [0, 100 * slope, -100 * slope, 0]], dtype=torch.float64)
    if kind == "sigmoid":
        want[0] = B.route_backward(x.double(), ids, dw.double(), kind, True, 1.0)[0]
    assert (got.cpu().double() - want).abs().max() < 100 * (2 * 100 + 96) * U


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_absent_experts_among_the_ids_have_no_part(cuda_device, kind, renorm):
    """An id whose logit is -inf or NaN counts as an empty slot, whatever its gradient."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(6, 40, generator=gen)
    ids = torch.stack([torch.randperm(40, generator=gen)[:6] for _ in range(6)]).int()
    dw = torch.randn(6, 6, generator=gen)
    empty = ids.clone()
    for t in range(6):
        x[t, ids[t, t]] = -INF if t % 2 else NAN
        dw[t, t] = NAN if t < 3 else INF
        empty[t, t] = -1
    args = dict(scores=kind, renormalize=renorm)
    got = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device), dw.to(cuda_device), **args)
    ref = tkq.route_topk_backward(x.to(cuda_device), empty.to(cuda_device), dw.to(cuda_device), **args)
    assert torch.isfinite(got).all() and torch.equal(got, ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(24, 5, 1), (64, 4, 4), (256, 8, 8), (1000, 32, 1)])
def test_weights_of_tiny_scores(cuda_device, dtype, kind, E, k, groups):
    """Experts chosen by their bias: weights are ratios of scores that are subnormal or no number."""
    T = 29
    x, gen = _low(T, E, 3 * E + k, dtype)
    x[3::8] = -INF                                # rows without experts next to them
    x[5::8, k // 2 + E // 2:] = -INF              # and rows with fewer than k low ones
    bias = torch.zeros(E)
    low = torch.randperm(E - E // 4, generator=gen) + E // 4
    bias[low] = 4.0 + torch.arange(len(low)).float() * 2.0 ** -6     # any two keys far apart
    ids, w = tkq.route_topk(x.to(cuda_device), k, kind, bias.to(cuda_device), num_groups=groups,
                            topk_groups=groups, scale=2.5)
    ref_ids, ref_w = B.route(x.double(), k, kind, bias.double(), groups=groups, topk_groups=groups, scale=2.5)
    full = (ref_ids >= E // 4).all(1) | (ref_ids < 0).all(1)         # no expert near 0 among the chosen
    assert full.sum() > T // 2
    assert torch.equal(ids.cpu()[full], ref_ids[full])
    tol = ((2 * _spread(x) + 64) * U * ref_w + 2.0 ** -60)
    assert (w.cpu().double() - ref_w)[full].abs().le(tol[full]).all()
    # a row's result does not depend on the rows that share its warp
    for t in range(T):
        a, b = tkq.route_topk(x[t:t + 1].to(cuda_device), k, kind, bias.to(cuda_device),
                              num_groups=groups, topk_groups=groups, scale=2.5)
        assert torch.equal(a[0], ids[t]) and torch.equal(b[0], w[t])


def test_lowest_finite_logits_are_experts_that_are_there(cuda_device):
    """The type's lowest value in the place of -inf: all experts of a row alike share the weight, with
    either kind of score."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((3, 16), torch.finfo(dtype).min, dtype=dtype, device=cuda_device)
        for kind in ("softmax", "sigmoid"):
            ids, w = tkq.route_topk(x, 4, kind)
            assert ids.tolist() == [[0, 1, 2, 3]] * 3 and (w == 0.25).all()
            d = tkq.route_topk_backward(x, ids, torch.tensor([[1.0, 0, 0, 0]] * 3, device=cuda_device), kind)
            want = torch.tensor([0.1875] + [-0.0625] * 3 + [0.0] * 12, device=cuda_device)
            assert torch.equal(d.float(), want.expand(3, 16))
