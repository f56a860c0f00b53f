"""The router's gradient in the example's training step with every product in FP8: the row weights' gradients come
back to their tokens from rows padded to groups of 128, against autograd in binary32.

The bound is that of test_gpu_moe_router with the casts of this path.  dw_e of a token is a sum over H of dy_c
silu(g_c) u_c.  g and u pass three casts each: the input, w1, the checkpoint; dy two: the rows of the gradient and
w2.  Each is off by at most 3.6 % in the root mean square, independent of the others, so a term is off by 3.6 %
sqrt(8) = 10.2 % of the root of the sum of squares n_e; weights from bf16 logits, bf16 products and the rounding of x
add less than 2 %.  So with m_e = w_e (n_e + sum_j w_j n_j) the error of the whole gradient is within 12.2 % of the root
of sum_t |x_t|^2 sum_e m_te^2."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from tests.test_gpu_moe_router import _norm

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,channels,hidden,experts,k", [
    (512, 512, 256, 8, 2), (301, 640, 384, 12, 4), (1, 256, 128, 4, 2), (64, 256, 128, 40, 3),
    (64, 256, 128, 40, 1)])
def test_router_gradient_with_fp8_products(cuda_device, tokens, channels, hidden, experts, k):
    import __graft_entry__
    __graft_entry__.build()
    import moe_block
    p = moe_block.parameters(channels, hidden, experts, cuda_device)
    gen = torch.Generator(device=cuda_device).manual_seed(7)
    r, h, gate, dr = ((torch.randn(tokens, channels, generator=gen, device=cuda_device) * s).bfloat16()
                      for s in (2.0, 1.0, 1.0, 0.1))
    _, saved = moe_block.forward(r, h, gate, p, k, 0.7, {n: moe_block.quantized(p[n]) for n in ("w1", "w2")})
    _, _, _, grads = moe_block.backward(dr, saved, p)

    ids = saved["ids"]
    leaf = p["router"].float().requires_grad_()
    f = {n: v.float() for n, v in p.items()}
    ref = moe_block.plain(r.float(), h.float(), gate.float(), {**f, "router": leaf}, ids, 0.7)
    ref.backward(dr.float())

    # the terms' magnitudes
    r1 = r.float() + 0.7 * _norm(h.float()) * f["w_post"] * torch.sigmoid(gate.float())
    x = _norm(r1) * f["w_pre"]
    shares = torch.softmax(x @ f["router"].t(), 1).gather(1, ids.long())
    w = shares / shares.sum(1, keepdim=True)
    acts, out = {}, torch.zeros_like(x)
    for e in range(experts):
        t, slot = (ids == e).nonzero(as_tuple=True)
        g, u = (x[t] @ f["w1"][e].t()).chunk(2, 1)
        acts[e] = t, slot, torch.nn.functional.silu(g) * u
        out.index_add_(0, t, acts[e][2] * w[t, slot, None] @ f["w2"][e].t())
    out.requires_grad_()
    dout, = torch.autograd.grad(_norm(out), out, dr.float())
    n = torch.zeros_like(w)
    for e, (t, slot, y) in acts.items():
        n[t, slot] = (dout[t] @ f["w2"][e] * y).norm(dim=1)
    m = w * (n + (w * n).sum(1, keepdim=True))
    bound = 0.122 * (x.square().sum(1) * m.square().sum(1)).sum().sqrt()

    err = (grads["router"].float() - leaf.grad).norm()
    assert err <= bound, (float(err), float(bound))
    if tokens == 512:                   # rows taken in another order would be off by the gradient itself
        assert leaf.grad.norm() > 2 * bound
