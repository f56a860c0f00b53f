"""Tiles of the products whose rows end inside a warp, one after another in one CTA: after each of them the warp's
lanes have parted, and the next tile's sums are read by all of them.  Whole numbers and scales of powers of two, so
every sum is exact."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def whole(shape, g, top=3):
    return torch.randint(-top, top + 1, shape, generator=g).float()


def powers(shape, g):
    return torch.randint(-2, 3, shape, generator=g).float().exp2()


@pytest.mark.parametrize("sms", [1, 2])
@pytest.mark.parametrize("sizes", [[1] * 9, [5, 31, 33, 64, 95, 0, 127, 128, 129, 1], [257, 3, 0, 0, 200]])
def test_rows_product(cuda_device, monkeypatch, sms, sizes):
    g = torch.Generator().manual_seed(len(sizes))
    E, N, K, dev = len(sizes), 384, 256, cuda_device
    offsets = torch.tensor([0] + sizes).cumsum(0).int()
    R = int(offsets[-1])
    a, w, a_sf, w_sf = whole((R, K), g), whole((E, N, K), g, 2), powers((R, K // 128), g), powers((E, N // 128, K // 128), g)
    want = experts64.product(a, a_sf, w, w_sf, offsets)[0].bfloat16()
    monkeypatch.setenv("TKQ_NUM_SMS", str(sms))
    for _ in range(3):
        got = tkq.expert_product(a.to(F8).to(dev), a_sf.to(dev), w.to(F8).to(dev), w_sf.to(dev), offsets.to(dev))
        assert torch.equal(got.cpu(), want)
    assert tkq.tkq_read_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient(cuda_device, monkeypatch, dtype):
    g = torch.Generator().manual_seed(4)
    groups, N, K, dev = [1, 0, 3, 2], 256, 384, cuda_device
    offsets = (torch.tensor([0] + groups).cumsum(0) * 128).int()
    R = int(offsets[-1])
    dy, x, dy_sf, x_sf = whole((N, R), g), whole((K, R), g), powers((N, R // 128), g), powers((K, R // 128), g)
    want = experts64.weight_grad(dy, dy_sf, x, x_sf, offsets)[0].to(dtype)
    monkeypatch.setenv("TKQ_NUM_SMS", "1")
    got = tkq.expert_weight_grad(dy.to(F8).to(dev), dy_sf.to(dev), x.to(F8).to(dev), x_sf.to(dev), offsets.to(dev),
                                 out_dtype=dtype)
    assert torch.equal(got.cpu(), want)
    assert tkq.tkq_read_device_status() == 0
