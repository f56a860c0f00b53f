"""Weights that are no numbers: a group of w4_cast that holds a NaN or an infinity has the scale NaN and codes
of zero, its neighbours are cast as without it, and a product with it is NaN."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def is_nan(sf):
    return sf == 255 if sf.dtype == torch.uint8 else sf.isnan()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("value", [NAN, -NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 31, 32, 127, 128, 200, 383])
def test_a_group_with_it_is_nan(cuda_device, group, value, at):
    N, K = 5, 384
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(at)).bfloat16()
    codes, sf = (t.cpu() for t in tkq.w4_cast(w.to(cuda_device), group))
    assert not bool(is_nan(sf).any())
    w[2, at] = value
    got, got_sf = (t.cpu() for t in tkq.w4_cast(w.to(cuda_device), group))
    bad = torch.zeros(N, K // group, dtype=torch.bool)
    bad[2, at // group] = True
    assert torch.equal(is_nan(got_sf), bad)
    assert torch.equal(got_sf[~bad], sf[~bad])
    cut = lambda c: c.view(N, K // group, group // 2)
    assert torch.equal(cut(got)[~bad], cut(codes)[~bad]) and not bool(cut(got)[bad].any())


@pytest.mark.parametrize("group", [32, 128])
def test_numbers_and_one_nan_among_all_lanes(cuda_device, group):
    """A NaN beside an infinity, beside zeros, and a whole group of them."""
    w = torch.zeros(4, 256, dtype=torch.bfloat16)
    w[0, 3], w[0, 4] = NAN, INF
    w[1, 255] = NAN
    w[2, :128] = NAN
    _, sf = tkq.w4_cast(w.to(cuda_device), group)
    bad = torch.zeros(4, 256 // group, dtype=torch.bool)
    bad[0, 0] = bad[1, -1] = True
    bad[2, :128 // group] = True
    assert torch.equal(is_nan(sf.cpu()), bad)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows,experts", [(1, 0), (5, 0), (40, 0), (6, 3)])
def test_products_with_it_are_nan(cuda_device, group, rows, experts):
    N, K = 128, 640
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(max(experts, 1), N, K, generator=g).bfloat16()
    x, xs = tkq.per_token_cast(torch.randn(rows, K, generator=g).bfloat16().to(cuda_device))
    x.view(torch.uint8)[0] = 0                       # a row of zeros: 0 NaN is NaN
    ids = torch.randint(0, experts, (rows, 2), dtype=torch.int32, generator=g) if experts else None
    product = lambda v: tkq.w4_product(x, xs, *tkq.w4_cast((v if experts else v[0]).to(cuda_device), group),
                                       None if ids is None else ids.to(cuda_device)).cpu()
    want = product(w)
    assert not bool(want.isnan().any())
    w[-1, 77, 600], w[-1, 3, 5] = NAN, INF
    got = product(w)
    bad = torch.zeros_like(want, dtype=torch.bool)
    hit = torch.ones(rows, dtype=torch.bool) if ids is None else ids.flatten() == experts - 1
    bad[hit.nonzero(), torch.tensor([3, 77])] = True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], want[~bad])
