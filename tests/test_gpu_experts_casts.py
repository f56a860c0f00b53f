"""The casts of expert_gather and expert_reduce_backward against their definition in elementary binary32
operations on the host: s = max(amax, 1e-4) / max and the codes of y / s, both IEEE quotients, tensor by tensor (a
division by a Python number may be done as a product with its rounded reciprocal, which moves a scale by its last
place and the quotients next to a tie with it).  Equal bit for bit."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def cast(v, fmt):
    dtype, top = FP8[fmt]
    g = v.view(v.shape[0], -1, 128)
    s = torch.maximum(g.abs().amax(2), torch.full((), 1e-4)) / torch.full((1, 1), top)
    return (g / s.unsqueeze(2)).view_as(v).to(dtype).view(torch.uint8), s


@pytest.mark.parametrize("T,k,E,C,align", [(4, 8, 256, 1408, 1), (333, 4, 12, 640, 128), (1000, 2, 8, 2048, 16)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_casts_are_the_quotients(cuda_device, T, k, E, C, align, fmt):
    g = torch.Generator().manual_seed(T)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.int()
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    x = torch.randn(T, C, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g) + 0.01
    order = tkq.expert_order(ids.to(cuda_device), E, align)
    pair = order.rows.cpu().long()
    live = pair >= 0
    pair = pair[live]
    codes, sf, _ = tkq.expert_gather(x.to(cuda_device), order, fmt)
    want, want_sf = cast(x.float(), fmt)
    assert torch.equal(sf.cpu()[live], want_sf[pair // k])
    assert torch.equal(codes.view(torch.uint8).cpu()[live], want[pair // k])
    y = torch.zeros(order.rows.numel(), C, dtype=torch.bfloat16, device=cuda_device)
    codes, sf, _ = tkq.expert_reduce_backward(x.to(cuda_device), y, order, w.to(cuda_device), fmt)
    want, want_sf = cast(w.flatten()[pair].unsqueeze(1) * x[pair // k].float(), fmt)
    assert torch.equal(sf.cpu()[live], want_sf)
    assert torch.equal(codes.view(torch.uint8).cpu()[live], want)
