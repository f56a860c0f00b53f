"""The block norms' gradients where a factor 1 / sqrt(mean) is very large or very small.

eps = 0 is accepted, so a row of h whose root mean square is 1e-14 has the factor 1e14: a product of
three of them is no binary32 number, while the gradients, p times sums of order one, are.  Bounds: those
of test_gpu_residual_norm, which are relative to the magnitudes of the terms."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests.test_gpu_residual_norm import BF, _backward_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


SCALES = [1.0, 1e-13, 1e-14, 3e-16, 1e-18, 1e10, 1e13, 1e15]


# one instance of each way to hold a row
@pytest.mark.parametrize("C", [640, 4224, 7168, 16384])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_any_magnitude(cuda_device, C, f32, gated):
    gen = torch.Generator().manual_seed(C)
    T, a = len(SCALES), 0.6
    s = torch.tensor(SCALES)[:, None]
    host = dict(r=torch.randn(T, C, generator=gen) * 3, h=(torch.randn(T, C, generator=gen) * s).bfloat16(),
                gate=torch.randn(T, C, generator=gen).bfloat16() if gated else None,
                w_post=1 + 0.3 * torch.randn(C, generator=gen), w_pre=1 + 0.3 * torch.randn(C, generator=gen))
    if not f32:
        host["r"] = host["r"].bfloat16()
    dev = {n: None if v is None else v.to(cuda_device) for n, v in host.items()}
    dr = torch.randn(T, C, generator=gen).to(host["r"].dtype)
    dx = (torch.randn(T, C, generator=gen) * 0.5).bfloat16()
    r1, _, _, _, p, q = tkq.residual_norm_and_cast(**dev, res_scale=a, eps=0.0)
    got = tkq.residual_norm_backward(dr.to(cuda_device), r1, dev["h"], dx.to(cuda_device), dev["w_post"],
                                     dev["gate"], dev["w_pre"], p, q, a)
    ref, bound = _backward_reference(host, dr.double(), dx.double(), r1.cpu().double(), p.cpu().double(),
                                     q.cpu().double(), a)
    rounds = (0 if f32 else BF, BF, BF, 0, 0)
    for name, t, g, b, rnd in zip(("dr", "dh", "dgate", "dw_post", "dw_pre"), got, ref, bound, rounds):
        if t is None:
            assert name == "dgate" and not gated
            continue
        assert torch.isfinite(t).all(), name
        err = (t.cpu().double() - g).abs()
        assert err.le(rnd * g.abs() + 1.01 * b).all(), (name, float((err / (rnd * g.abs() + b)).max()))
