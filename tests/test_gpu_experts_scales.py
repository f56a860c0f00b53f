"""The scales that expert_reduce_backward writes beside a cast: those of rows with a pair as per_token_cast writes them,
the smallest scale fl(1e-4 / max) at rows that pad an expert's, and nothing behind the last expert's."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
GUARD = 7.0
TOP = {"e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("T,k,E,C,align", [(1, 1, 1, 128, 1), (4, 8, 256, 1408, 128), (33, 2, 7, 640, 16), (257, 6, 60, 384, 128),
                                           (130, 32, 40, 256, 1), (1000, 3, 5, 128, 128), (5, 8, 8, 2048, 3)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_of_every_row(cuda_device, T, k, E, C, align, fmt):
    g = torch.Generator().manual_seed(C + T)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.int()
    ids[torch.rand(T, k, generator=g) < 0.2] = -1
    order = tkq.expert_order(ids.to(cuda_device), E, align)
    R, end = order.rows.numel() + 7, int(order.offsets[-1])     # some rows behind the last expert's for certain
    order = tkq.expert_order(ids.to(cuda_device), E, align, rows=torch.empty(R, dtype=torch.int32, device=cuda_device))
    d, w = torch.randn(T, C, generator=g).bfloat16(), torch.randn(T, k, generator=g)
    y = torch.zeros(R, C, dtype=torch.bfloat16, device=cuda_device)
    out = torch.full((R, C), 0x55, dtype=torch.uint8, device=cuda_device)
    out_sf = torch.full((R, C // 128), GUARD, device=cuda_device)
    dy, sf, _ = tkq.expert_reduce_backward(d.to(cuda_device), y, order, w.to(cuda_device), fmt, out=out, out_sf=out_sf)
    assert dy is out and sf is out_sf
    pair = order.rows.cpu().long()
    live, behind = pair >= 0, torch.arange(R) >= end
    pad = ~live & ~behind
    codes, want = tkq.per_token_cast((w.unsqueeze(2) * d.float().unsqueeze(1)).view(T * k, C).to(cuda_device), fmt)
    sf, dy = sf.cpu(), dy.cpu()
    assert torch.equal(sf[live], want.cpu()[pair[live]]) and torch.equal(dy[live], codes.view(torch.uint8).cpu()[pair[live]])
    smallest = torch.tensor(1e-4) / torch.tensor(TOP[fmt])
    assert bool((sf[pad] == smallest).all()) and not bool(dy[pad].any())
    assert bool((sf[behind] == GUARD).all()) and bool((dy[behind] == 0x55).all())
    assert bool(pad.any()) or align < 16
