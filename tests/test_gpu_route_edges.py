"""Routing's edges: gradients that meet absent experts."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu

INF = float("inf")
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


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
