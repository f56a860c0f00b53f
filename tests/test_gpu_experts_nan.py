"""NaN and infinities in the operands of the experts' products: a NaN code or scale makes NaN of its own row or column of
its own expert and changes nothing else, bit for bit; so does an E5M2 infinity, whose products with zeros are NaN."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
F8, F8W = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def same_but(got, want, bad):
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], want[~bad])


def with_value(t, at, value):
    t = t.clone()
    t.view(torch.uint8)[at] = value
    return t


def with_scale(t, at, value):
    t = t.clone()
    t[at] = value
    return t


def test_rows_product(cuda_device):
    g = torch.Generator().manual_seed(1)
    sizes, N, K = [70, 0, 130, 33], 384, 256
    offsets = torch.tensor([0] + sizes).cumsum(0).int()
    R, E = int(offsets[-1]), len(sizes)
    codes = lambda *s: torch.randn(*s, generator=g).to(F8).to(cuda_device)
    a, w = codes(R, K), torch.randn(E, N, K, generator=g).to(F8W).to(cuda_device)
    a_sf, w_sf = (torch.rand(*s, generator=g).to(cuda_device) for s in ((R, K // 128), (E, N // 128, K // 128)))
    a.view(torch.uint8)[5] = 0
    run = lambda a, a_sf, w, w_sf: tkq.expert_product(a, a_sf, w, w_sf, offsets.to(cuda_device)).cpu()
    want = run(a, a_sf, w, w_sf)
    assert not bool(want.isnan().any())
    none = torch.zeros(R, N, dtype=torch.bool)
    for r in (0, 5, 69, 70, R - 1):                  # the first and last rows of experts
        bad = none.clone()
        bad[r] = True
        same_but(run(with_value(a, (r, 200), 0x7F), a_sf, w, w_sf), want, bad)
        same_but(run(a, with_scale(a_sf, (r, 1), NAN), w, w_sf), want, bad)
    for e, n in ((0, 0), (2, 383), (3, 128)):
        bad = none.clone()
        bad[int(offsets[e]):int(offsets[e + 1]), n] = True
        same_but(run(a, a_sf, with_value(w, (e, n, 3), 0x7F), w_sf), want, bad)
        bad[int(offsets[e]):int(offsets[e + 1]), n // 128 * 128:n // 128 * 128 + 128] = True
        same_but(run(a, a_sf, w, with_scale(w_sf, (e, n // 128, 0), NAN)), want, bad)
    # an infinity times the zeros of row 5 is NaN, times anything else infinite
    got = run(a, a_sf, with_value(w, (0, 7, 9), 0x7C), w_sf)
    bad = none.clone()
    bad[:70, 7] = True
    assert bool(got[5, 7].isnan()) and not bool(got[:70, 7].isfinite().any()) and torch.equal(got[~bad], want[~bad])


def test_weight_gradient(cuda_device):
    g = torch.Generator().manual_seed(2)
    offsets = torch.tensor([0, 128, 128, 512, 640], dtype=torch.int32)
    R, N, K, E = 768, 256, 384, 4                    # the last group of rows is no expert's
    codes = lambda *s: torch.randn(*s, generator=g).to(F8).to(cuda_device)
    dy, x = codes(N, R), codes(K, R)
    dy_sf, x_sf = (torch.rand(*s, generator=g).to(cuda_device) for s in ((N, R // 128), (K, R // 128)))
    run = lambda dy, dy_sf, x, x_sf: tkq.expert_weight_grad(dy, dy_sf, x, x_sf, offsets.to(cuda_device)).cpu()
    want = run(dy, dy_sf, x, x_sf)
    none = torch.zeros(E, N, K, dtype=torch.bool)
    assert not bool(want.isnan().any())
    for r, e in ((0, 0), (127, 0), (128, 2), (511, 2), (512, 3), (639, 3), (640, None), (767, None)):
        for n in (0, 255):
            bad = none.clone()
            if e is not None:
                bad[e, n] = True
            same_but(run(with_value(dy, (n, r), 0x7F), dy_sf, x, x_sf), want, bad)
            same_but(run(dy, with_scale(dy_sf, (n, r // 128), NAN), x, x_sf), want, bad)
        for k in (0, 383):
            bad = none.clone()
            if e is not None:
                bad[e, :, k] = True
            same_but(run(dy, dy_sf, with_value(x, (k, r), 0xFF), x_sf), want, bad)
            same_but(run(dy, dy_sf, x, with_scale(x_sf, (k, r // 128), NAN)), want, bad)


@pytest.mark.parametrize("group", [32, 128])
def test_4_bit_product(cuda_device, group):
    g = torch.Generator().manual_seed(3)
    T, N, K, E = 21, 128, 640, 3
    x = torch.randn(T, K, generator=g).to(F8).to(cuda_device)
    xs = torch.rand(T, K // 128, generator=g).to(cuda_device)
    w, ws = tkq.w4_cast(torch.randn(E, N, K, generator=g).bfloat16().to(cuda_device), group)
    ids = torch.randint(0, E, (T, 2), dtype=torch.int32, generator=g)
    run = lambda x, xs: tkq.w4_product(x, xs, w, ws, ids.to(cuda_device)).cpu()
    want = run(x, xs)
    for t in (0, 8, 20):
        bad = torch.zeros(2 * T, N, dtype=torch.bool)
        bad[2 * t:2 * t + 2] = True
        same_but(run(with_value(x, (t, 639), 0x7F), xs), want, bad)
        same_but(run(x, with_scale(xs, (t, 4), NAN)), want, bad)
