"""One training step of a mixture-of-experts block around this library's calls.

Forward: the norm after the block before and the norm before this one, in one
pass that ends in the FP8 cast; routing; the tokens' rows in the order of their
experts; the experts' SwiGLU fused with its cast and an 8-bit checkpoint of its
input; the sum of each token's rows.  Backward: the SwiGLU from the checkpoint,
with the gradient of the routing weights and the activations that the last weight
gradient needs; the routing's gradient; the norms' gradients.  The products are
PyTorch's (one per expert, bf16), or with --fp8 the library's of FP8 codes and
scales, weight gradients included: then nothing waits for the host.

    python examples/moe_block.py [--tokens 4096] [--channels 2048] [--hidden 1408]
                                 [--experts 64] [--topk 6] [--fp8]

prints how far the outputs and gradients are from the same block in binary32
without any quantization, and what the checkpoint holds.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_activation_quantization_gb300 as tkq  # noqa: E402


def parameters(channels, hidden, experts, device, seed=0):
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device=device) * std).bfloat16()
    return dict(w_post=torch.ones(channels, device=device), w_pre=torch.ones(channels, device=device),
                router=normal(experts, channels, std=channels ** -0.5),
                w1=normal(experts, 2 * hidden, channels, std=channels ** -0.5),
                w2=normal(experts, channels, hidden, std=hidden ** -0.5))


def expert_products(x, weights, sizes):
    """x [rows, a] grouped by expert times weights [experts, b, a], expert by expert."""
    return torch.cat([part @ w.t() for part, w in zip(x.split(sizes), weights)])


def weight_products(dy, x, sizes):
    return torch.stack([a.t() @ b for a, b in zip(dy.split(sizes), x.split(sizes))])


def quantized(weights):
    """Codes and block scales of [experts, b, a] matrices, and of their transposes: what the FP8
    products read forward and backward, made once after each update of the weights."""
    experts, b, a = weights.shape
    codes, sf = zip(*(tkq.per_block_cast(w) for w in weights))
    codes, sf = torch.stack([c.view(torch.uint8) for c in codes]), torch.stack(sf)
    t_codes, t_sf = codes.transpose(1, 2).contiguous(), sf.transpose(1, 2).contiguous()
    return tuple(v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v for v in (codes, sf, t_codes, t_sf))


def forward(r, h, gate, p, k, res_scale=1.0, fp8=None):
    """The residual stream after the block, and what the backward needs.  fp8: the quantized w1 and w2, or
    None for PyTorch's products."""
    r1, xq, xs, x, post, pre = tkq.residual_norm_and_cast(
        r, h, w_post=p["w_post"], gate=gate, w_pre=p["w_pre"], res_scale=res_scale, with_bf16=True)
    logits = x @ p["router"].t()
    counts = torch.zeros(len(p["router"]), dtype=torch.int32, device=r.device)
    ids, weights = tkq.route_topk(logits, k, scores="softmax", counts=counts)
    # rows of the experts' products: (token, slot) pairs in the order of their experts, each expert's
    # padded to groups of 128 where the weight gradients sum over such groups
    order = tkq.expert_order(ids, len(p["w1"]), align=128 if fp8 else 1)
    rows_q, rows_s, w = tkq.expert_gather(xq, order, x_sf=xs, weights=weights)
    if fp8:
        sizes = None
        z = tkq.expert_product(rows_q, rows_s, *fp8["w1"][:2], order.offsets)
    else:
        sizes = counts.tolist()
        z = expert_products(tkq.cast_back(rows_q, rows_s, out_dtype=torch.bfloat16), p["w1"], sizes)
    yq, ys, ckpt, ckpt_sf = tkq.swiglu_forward_cast_and_checkpoint(z, topk_weights=w)
    if fp8:
        rows = tkq.expert_product(yq, ys, *fp8["w2"][:2], order.offsets)
    else:
        rows = expert_products(tkq.cast_back(yq, ys, out_dtype=torch.bfloat16), p["w2"], sizes)
    out, _ = tkq.expert_reduce(rows, order)
    r2, _, _, _, post2, _ = tkq.residual_norm_and_cast(r1, out, fmt=None)
    saved = dict(r1=r1, h=h, gate=gate, x=x, post=post, pre=pre, logits=logits, ids=ids, order=order, w=w,
                 sizes=sizes, inputs=(rows_q, rows_s), ckpt=ckpt, ckpt_sf=ckpt_sf, out=out, post2=post2,
                 res_scale=res_scale, k=k, fp8=fp8)
    return r2, saved


def backward(dr, s, p):
    """Gradients of the stream, the block before's output, its gate, and the parameters."""
    dr1, dout, _, _, _ = tkq.residual_norm_backward(dr, None, s["out"], rstd_post=s["post2"])
    order, sizes, fp8 = s["order"], s["sizes"], s["fp8"]
    rows, _, _ = tkq.expert_gather(dout, order)
    if fp8:
        dq, dsf, _ = tkq.expert_gather(dout, order, fmt="e4m3")
        dy = tkq.expert_product(dq, dsf, *fp8["w2"][2:], order.offsets)
    else:
        dy = expert_products(rows, p["w2"].transpose(1, 2), sizes)
    dz, _, dw, y = tkq.swiglu_backward_from_checkpoint(s["ckpt"], s["ckpt_sf"], dy, topk_weights=s["w"],
                                                       with_weight_grad=True, with_y=True)
    inputs = tkq.cast_back(*s["inputs"], out_dtype=torch.bfloat16)
    if fp8:
        def weight_grad(d, v):
            return tkq.expert_weight_grad(*tkq.per_channel_cast(d, transpose=True),
                                          *tkq.per_channel_cast(v, transpose=True), order.offsets)
        grads = dict(w2=weight_grad(rows, y), w1=weight_grad(dz, inputs))
        dx_rows = tkq.expert_product(*tkq.per_token_cast(dz), *fp8["w1"][2:], order.offsets)
    else:
        grads = dict(w2=weight_products(rows, y, sizes), w1=weight_products(dz, inputs, sizes))
        dx_rows = expert_products(dz, p["w1"].transpose(1, 2), sizes)
    # back at their tokens: the rows' gradients added up, those of the routing weights in their places
    dx, dweights = tkq.expert_reduce(dx_rows, order, row_values=dw, out_dtype=torch.float32)
    dlogits = tkq.route_topk_backward(s["logits"], s["ids"], dweights, scores="softmax")
    grads["router"] = dlogits.t() @ s["x"]
    dx += dlogits @ p["router"]
    d, dh, dgate, grads["w_post"], grads["w_pre"] = tkq.residual_norm_backward(
        dr1, s["r1"], s["h"], dx=dx.bfloat16(), w_post=p["w_post"], gate=s["gate"], w_pre=p["w_pre"],
        rstd_post=s["post"], rstd_pre=s["pre"], res_scale=s["res_scale"])
    return d, dh, dgate, grads


def plain(r, h, gate, p, ids, res_scale=1.0, eps=1e-6):
    """The same block in binary32 with the same choice of experts, for autograd."""
    def norm(v):
        return v * (v.square().mean(1, keepdim=True) + eps).rsqrt()
    r1 = r + res_scale * norm(h) * p["w_post"] * torch.sigmoid(gate)
    x = norm(r1) * p["w_pre"]
    shares = torch.softmax(x @ p["router"].t(), 1).gather(1, ids.long())
    weights = shares / shares.sum(1, keepdim=True)
    out = torch.zeros_like(r)
    for e in range(len(p["w1"])):
        t, slot = (ids == e).nonzero(as_tuple=True)
        g, u = (x[t] @ p["w1"][e].t()).chunk(2, 1)
        y = torch.nn.functional.silu(g) * u * weights[t, slot, None]
        out = out.index_add(0, t, y @ p["w2"][e].t())
    return r1 + norm(out)


def step(tokens, channels, hidden, experts, k, device="cuda", seed=1, fp8=False):
    """One step through the library and one through autograd: {name: relative 2-norm error}."""
    p = parameters(channels, hidden, experts, device)
    gen = torch.Generator(device=device).manual_seed(seed)
    r, h, gate, dr = ((torch.randn(tokens, channels, generator=gen, device=device) * s).bfloat16()
                      for s in (2.0, 1.0, 1.0, 0.1))
    r2, saved = forward(r, h, gate, p, k, 0.7, {n: quantized(p[n]) for n in ("w1", "w2")} if fp8 else None)
    d, dh, dgate, grads = backward(dr, saved, p)

    leaves = [t.float().requires_grad_() for t in (r, h, gate)]
    params = {n: v.float().requires_grad_() for n, v in p.items()}
    ref = plain(*leaves, params, saved["ids"], 0.7)
    ref.backward(dr.float())
    pairs = {"stream": (r2, ref), "d stream": (d, leaves[0].grad), "d h": (dh, leaves[1].grad),
             "d gate": (dgate, leaves[2].grad)}
    pairs.update({f"d {n}": (grads[n], params[n].grad) for n in grads})
    errors = {n: float((a.float() - b.detach()).norm() / b.detach().norm()) for n, (a, b) in pairs.items()}
    return errors, saved


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--channels", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--fp8", action="store_true", help="the experts' products in FP8")
    a = ap.parse_args()
    errors, saved = step(a.tokens, a.channels, a.hidden, a.experts, a.topk, fp8=a.fp8)
    for name, e in errors.items():
        print(f"{name:12s} {100 * e:6.2f} % from binary32 without quantization")
    held = saved["ckpt"].numel() + 4 * saved["ckpt_sf"].numel()
    print(f"checkpoint of the SwiGLU's input: {held / 1e6:.1f} MB, {2 * saved['ckpt'].numel() / 1e6:.1f} MB in bf16")


if __name__ == "__main__":
    main()
