"""The weight gradient in a captured graph behind the calls that give its operands, replayed on inputs whose offsets,
rows and gradients are others: it is that of the eager calls, differs from seed to seed, and is within its
64-bit formula's bound.

Bound: the one of test_gpu_experts (u = 2^-24): (4 x 33 x 2 + 3 + groups) u of the sum of magnitudes."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T, k, E, C, N = 300, 4, 6, 384, 256


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def fresh(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    liking = torch.randn(E, generator=g, device="cuda") * 2
    ids = (liking + torch.rand(T, E, generator=g, device="cuda")).topk(k, 1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids)
    return (ids.contiguous(), torch.randn(T, C, generator=g, device="cuda").bfloat16(),
            torch.randn(T, N, generator=g, device="cuda").bfloat16())


def chain(ids, x, d, dtype):
    order = tkq.expert_order(ids, E)
    R = order.rows.numel()
    zeros = lambda width: torch.zeros(R, width, dtype=torch.bfloat16, device="cuda")
    xr, _, _ = tkq.expert_gather(x, order, out=zeros(C))
    dr, _, _ = tkq.expert_gather(d, order, out=zeros(N))
    operands = *tkq.per_channel_cast(dr, "e5m2", transpose=True), *tkq.per_channel_cast(xr, transpose=True)
    return order.offsets, *operands, tkq.expert_weight_grad(*operands, order.offsets, out_dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_weight_gradient(cuda_device, dtype):
    held = [t.clone() for t in fresh(1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*held, dtype)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(*held, dtype)
    seen, starts = [], []
    for seed in (2, 3, 4, 2):
        for to, new in zip(held, fresh(seed)):
            to.copy_(new)
        want = [t.clone() for t in chain(*held, dtype)]
        for _ in range(2):
            outs[-1].fill_(float("nan"))
            graph.replay()
            for i, (a, b) in enumerate(zip(outs, want)):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i
        offsets, dy_t, dy_sf, x_t, x_sf, dw = (t.cpu() for t in outs)
        ref, size = experts64.weight_grad(dy_t.float(), dy_sf, x_t.float(), x_sf, offsets)
        bound = (4 * 33 * 2 + 3 + int(offsets.diff().max()) // 128) * U * size
        if dtype is torch.bfloat16:
            bound = bound + 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs()
        assert bool(((dw.double() - ref).abs() <= bound).all())
        assert bool((ref != 0).any(2).any(1)[offsets.diff() > 0].all()) and bool(dw.any())
        seen.append(dw.clone())
        starts.append(offsets.tolist())
    assert torch.equal(seen[0], seen[3])
    assert starts[0] != starts[1] and not any(torch.equal(a, b) for a, b in ((seen[0], seen[1]), (seen[1], seen[2])))
    assert tkq.tkq_read_device_status() == 0
