"""What the operators around an FP8 block are measured on: expert routing, the SwiGLU with an 8-bit
checkpoint, and the norms around a block, each in its forward and its backward direction.

``own`` False computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end); ``own`` True makes the calls a user makes of this package.  FP8 outputs are returned as
float8 tensors, which hold the values their codes stand for, beside their fp32 scales.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = 128
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = float(torch.finfo(torch.float32).max)


def listed():
    return [
        # a decoding step of a few sequences: 256 experts in 8 groups of which 4 are searched, sigmoid
        # scores with a bias for balance; latency counts
        dict(name="route, 3 tokens", op="route", T=3, E=256, k=8, dtype="f32", scores="sigmoid", bias=True,
             groups=8, topk_groups=4, renorm=True, scale=2.5, masked=False),
        # the same router over a prompt or a training batch of 16384 tokens
        dict(name="route, 16384 tokens", op="route", T=16384, E=256, k=8, dtype="f32", scores="sigmoid",
             bias=True, groups=8, topk_groups=4, renorm=True, scale=2.5, masked=False),
        # a small training batch of odd sizes, softmax over 60 experts, bf16 logits, padding tokens
        # whose logits are all -inf
        dict(name="route backward, 1021 tokens", op="route_bwd", T=1021, E=60, k=4, dtype="bf16",
             scores="softmax", renorm=False, scale=1.0, masked=True),
        # the backward of the large router, softmax with renormalised weights
        dict(name="route backward, 16384 tokens", op="route_bwd", T=16384, E=256, k=8, dtype="f32",
             scores="softmax", renorm=True, scale=2.5, masked=False),
        # the rows one expert gets from a small batch: SwiGLU, cast and checkpoint, odd sizes
        dict(name="save, 77 rows", op="save", T=77, H=1408, fmt="e4m3", ckpt_fmt="e4m3", weighted=True),
        # 8192 tokens sent to 8 experts each, H = 2048: the forward of all experts' SwiGLU in one call
        dict(name="save, 65536 rows", op="save", T=65536, H=2048, fmt="e4m3", ckpt_fmt="e4m3", weighted=True),
        # the backward of a shared expert on an odd batch: bf16 gradients, no routing weight
        dict(name="restore, 1531 rows", op="restore", T=1531, H=1408, fmt="bf16", ckpt_fmt="e5m2",
             weighted=False, y=False),
        # the backward of the 65536 rows: FP8 gradients for the next products, the gradient of the
        # routing weights, and y again for the weight gradient of the product that follows
        dict(name="restore, 65536 rows", op="restore", T=65536, H=2048, fmt="e4m3", ckpt_fmt="e4m3",
             weighted=True, y=True),
        # one token of each of 4 sequences: post-norm with gate, residual, pre-norm, cast for the FP8 product
        dict(name="norm, 4 tokens", op="norm", T=4, C=7168, residual="bf16", post=True, gate=True, pre=True,
             fmt="e4m3", bf16=False),
        # the same over a batch of 8192 tokens
        dict(name="norm, 8192 tokens", op="norm", T=8192, C=7168, residual="bf16", post=True, gate=True,
             pre=True, fmt="e4m3", bf16=False),
        # an odd batch with the residual stream in 32 bits and no gate
        dict(name="norm backward, 777 tokens", op="norm_bwd", T=777, C=2176, residual="f32", post=True,
             gate=False, pre=True),
        # training on 8192 tokens: all gradients of the block's norms, gate and residual
        dict(name="norm backward, 8192 tokens", op="norm_bwd", T=8192, C=7168, residual="bf16", post=True,
             gate=True, pre=True),
    ]


def draw(rng):
    def size(lo, hi):
        n = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))
        return n + 1 if n == 3072 else n

    def width(most):
        n = size(1, most)
        return GROUP * (n + 1 if n in (12, 24) else n)

    op = rng.choice(["route", "route_bwd", "save", "restore", "norm", "norm_bwd"])
    if op in ("route", "route_bwd"):
        c = dict(op=op, dtype=rng.choice(["bf16", "f32"]), scores=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.4)
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        c["E"] = groups * size(max(1, 8 // groups), 512 // groups)
        c["k"] = rng.randint(1, min(c["E"], 16))
        if op == "route":
            c.update(bias=rng.random() < 0.6, groups=groups, topk_groups=rng.randint(1, groups))
        c["T"] = size(1, min(32768, 16384 * 256 // c["E"]))
    elif op in ("save", "restore"):
        c = dict(op=op, H=width(64), ckpt_fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                 weighted=rng.random() < 0.6)
        c["T"] = size(1, min(65536, 65536 * 2048 // c["H"]))
        if op == "save":
            c.update(fmt=rng.choice(["e4m3", "e4m3", "e5m2"]))
        else:
            c.update(fmt=rng.choice(["bf16", "e4m3", "e5m2"]), y=rng.random() < 0.5)
    else:
        c = dict(op=op, C=width(64), residual=rng.choice(["bf16", "f32"]), post=rng.random() < 0.7,
                 gate=rng.random() < 0.5, pre=rng.random() < 0.85)
        c["T"] = size(1, min(32768, 8192 * 7168 // c["C"] // (2 if c["residual"] == "f32" else 1)))
        if op == "norm":
            c.update(fmt=rng.choice(["e4m3", "e5m2", "none"]) if c["pre"] else "none")
            c.update(bf16=c["pre"] and (c["fmt"] == "none" or rng.random() < 0.3))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)


def _logits(gen, T, E, case):
    x = torch.randn(T, E, generator=gen, device=DEV) * 1.5
    if case["masked"]:  # a few experts taken from a few tokens; every 16th token is padding
        x = x.masked_fill(torch.rand(T, E, generator=gen, device=DEV) < 0.05, -math.inf)
        x[::16] = -math.inf
    return x.to(DTYPES[case["dtype"]])


def _undecided(x, bias, case):
    """Rows in which two experts or two groups next to one another in the order are nearer than the last
    bits of a 32-bit score, without being equal: either order is right there, so such rows are drawn
    again and whole numbers can be compared."""
    x64, T, E = x.double(), x.shape[0], x.shape[1]
    live = x64 > -math.inf
    if case["scores"] == "sigmoid":
        key = torch.sigmoid(x64)
    else:
        key = torch.softmax(torch.where(live, x64, -1e30), 1)
    key = torch.where(live, key + (0 if bias is None else bias.double()), -math.inf)
    if case["groups"] > 1:
        per = key.view(T, case["groups"], -1)
        two = per.topk(min(2, per.shape[2]), 2).values
        of_group = torch.where(two > -math.inf, two, 0).sum(2).masked_fill(two[:, :, 0] == -math.inf, -math.inf)
        lists = [per.flatten(1), of_group]
    else:
        lists = [key]
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    for v in lists:
        v = v.sort(1, descending=True).values
        gap = v[:, :-1] - v[:, 1:]
        near = (gap > 0) & (gap < 3e-6 * v[:, :-1].abs())
        # without groups only the first k and the one after them are looked at
        bad |= near[:, :case["k"]].any(1) if case["groups"] == 1 else near.any(1)
    return bad


def _quantized(x, fmt):
    """Codes and scales of 1x128 groups of an fp32 matrix."""
    dtype, top = FP8[fmt]
    v = x.view(x.shape[0], -1, GROUP)
    s = v.abs().amax(2).clamp_min(1e-4) / top
    return (v / s.unsqueeze(2)).view_as(x).to(dtype), s


def prepare(case, seed):
    gen, T, op = _generator(seed), case["T"], case["op"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = dict(case)
    if op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        x = _logits(gen, T, E, case)
        if op == "route":
            bias = normal(E, std=0.03 if case["scores"] == "sigmoid" else 0.3 / E, dtype=torch.float32) if case["bias"] else None
            for _ in range(20):
                bad = _undecided(x, bias, case)
                if not bool(bad.any()):
                    break
                x = torch.where(bad.unsqueeze(1), _logits(gen, T, E, case), x)
            s.update(logits=x, bias=bias)
        else:
            top = x.float().topk(k, 1)
            s.update(logits=x, ids=torch.where(top.values > -math.inf, top.indices, -1).int(),
                     dweights=normal(T, k, dtype=torch.float32))
    elif op == "save":
        H = case["H"]
        s.update(x=torch.cat([normal(T, H, std=2.0), normal(T, H)], 1))
    elif op == "restore":
        H = case["H"]
        s["ckpt"], s["ckpt_sf"] = _quantized(torch.cat([normal(T, H, std=2.0), normal(T, H)], 1).float(), case["ckpt_fmt"])
        s["dy"] = normal(T, H, std=0.5)
    else:
        C = case["C"]
        res = DTYPES[case["residual"]]
        s["h"] = normal(T, C, std=0.7)
        s["w_post"] = 1 + normal(C, std=0.2, dtype=torch.float32)
        s["gate"] = normal(T, C) if case["gate"] else None
        s["w_pre"] = 1 + normal(C, std=0.2, dtype=torch.float32) if case["pre"] else None
        s["r"] = normal(T, C, std=3.0, dtype=res)
        s["res_scale"], s["eps"] = 0.7, 1e-6
        if op == "norm_bwd":
            # what the forward left behind: r is the stream after the block here
            s["rstd_post"] = (s["h"].float().square().mean(1) + s["eps"]).rsqrt() if case["post"] else None
            s["rstd_pre"] = (s["r"].float().square().mean(1) + s["eps"]).rsqrt() if case["pre"] else None
            s["dx"] = normal(T, C, std=0.5) if case["pre"] else None
            s["dr"] = normal(T, C, std=0.5, dtype=res)
    if op in ("save", "restore"):
        s["w"] = (torch.rand(T, generator=gen, device=DEV) * 0.3 + 0.01) if case["weighted"] else None
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


def _own(s):
    import fp8_activation_quantization_gb300 as tkq
    op = s["op"]
    if op == "route":
        counts = torch.zeros(s["E"], dtype=torch.int32, device=DEV)
        ids, weights = tkq.route_topk(s["logits"], s["k"], scores=s["scores"], bias=s["bias"],
                                      num_groups=s["groups"], topk_groups=s["topk_groups"],
                                      renormalize=s["renorm"], scale=s["scale"], counts=counts)
        return ids, weights, counts
    if op == "route_bwd":
        return tkq.route_topk_backward(s["logits"], s["ids"], s["dweights"], scores=s["scores"],
                                       renormalize=s["renorm"], scale=s["scale"])
    if op == "save":
        return tkq.swiglu_forward_cast_and_checkpoint(s["x"], s["fmt"], topk_weights=s["w"],
                                                      ckpt_fmt=s["ckpt_fmt"])
    if op == "restore":
        return tkq.swiglu_backward_from_checkpoint(s["ckpt"], s["ckpt_sf"], s["dy"],
                                                   None if s["fmt"] == "bf16" else s["fmt"],
                                                   topk_weights=s["w"], with_weight_grad=s["weighted"],
                                                   with_y=s["y"])
    if op == "norm":
        return tkq.residual_norm_and_cast(s["r"], s["h"], w_post=s["w_post"], gate=s["gate"],
                                          w_pre=s["w_pre"], post_norm=s["post"], res_scale=s["res_scale"],
                                          eps=s["eps"], fmt=None if s["fmt"] == "none" else s["fmt"],
                                          with_bf16=s["bf16"])
    return tkq.residual_norm_backward(s["dr"], s["r"], s["h"], dx=s["dx"], w_post=s["w_post"],
                                      gate=s["gate"], w_pre=s["w_pre"], rstd_post=s["rstd_post"],
                                      rstd_pre=s["rstd_pre"], res_scale=s["res_scale"])


def _plain_scores(x, kind):
    x = x.float()
    live = x > -math.inf
    x = x.clamp(max=LARGEST)
    if kind == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        top = torch.where(live, x, -LARGEST).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(x - top), 0)
        score = e / e.sum(1, keepdim=True).clamp_min(1)
    return torch.where(live, score, 0), live


def _plain_route(s):
    T, E, k = s["T"], s["E"], s["k"]
    score, live = _plain_scores(s["logits"], s["scores"])
    key = torch.where(live, score if s["bias"] is None else score + s["bias"], -math.inf)
    if s["groups"] > 1:
        per = key.view(T, s["groups"], -1)
        two = per.topk(min(2, per.shape[2]), 2).values
        of_group = torch.where(two > -math.inf, two, 0).sum(2).masked_fill(two[:, :, 0] == -math.inf, -math.inf)
        first = of_group.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        taken = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, first, True)
        key = torch.where(taken.unsqueeze(2), per, -math.inf).view(T, E)
    value, ids = key.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    chosen = value > -math.inf
    w = torch.where(chosen, score.gather(1, ids), 0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    ids = torch.where(chosen, ids, -1).int()
    slot = torch.where(chosen, ids, E).flatten()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=DEV).index_add_(0, slot, torch.ones_like(slot))
    return ids, w * s["scale"], counts[:E]


def _plain_route_bwd(s):
    score, live = _plain_scores(s["logits"], s["scores"])
    chosen = s["ids"] >= 0
    ids = torch.where(chosen, s["ids"], 0).long()
    picked = torch.where(chosen, score.gather(1, ids), 0)
    d = torch.where(chosen, s["dweights"], 0) * s["scale"]
    if s["renorm"]:
        total = picked.sum(1, keepdim=True)
        d = torch.where(total > 0, (d - (d * picked).sum(1, keepdim=True) / total) / total, 0)
    ds = torch.zeros_like(score).scatter_add_(1, ids, torch.where(chosen, d, 0))
    if s["scores"] == "sigmoid":
        e = torch.exp(-s["logits"].float().abs())
        dx = ds * e / (1 + e).square()
    else:
        dx = score * (ds - (ds * score).sum(1, keepdim=True))
    return torch.where(live, dx, 0).to(s["logits"].dtype)


def _plain_save(s):
    x = s["x"].float()
    g, u = x[:, :s["H"]], x[:, s["H"]:]
    y = g / (1 + torch.exp(-g)) * u
    if s["w"] is not None:
        y = y * s["w"].unsqueeze(1)
    return *_quantized(y.contiguous(), s["fmt"]), *_quantized(x, s["ckpt_fmt"])


def _plain_restore(s):
    T, H = s["T"], s["H"]
    x = (s["ckpt"].float().view(T, -1, GROUP) * s["ckpt_sf"].unsqueeze(2)).view(T, 2 * H)
    g, u, d = x[:, :H], x[:, H:], s["dy"].float()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    dw = (d * silu * u).sum(1) if s["weighted"] else None
    w = s["w"].unsqueeze(1) if s["weighted"] else 1.0
    dx = torch.cat([d * u * sig * (1 + g * (1 - sig)) * w, d * silu * w], 1)
    y = (silu * u * w).bfloat16() if s["y"] else None
    if s["fmt"] == "bf16":
        return dx.bfloat16(), None, dw, y
    return *_quantized(dx, s["fmt"]), dw, y


def _plain_norm(s):
    h = s["h"].float()
    p = (h.square().mean(1) + s["eps"]).rsqrt() if s["post"] else None
    b = (h if p is None else h * p.unsqueeze(1)) * s["w_post"]
    if s["gate"] is not None:
        b = b / (1 + torch.exp(-s["gate"].float()))
    r = s["r"].float() + s["res_scale"] * b
    if not s["pre"]:
        return r.to(s["r"].dtype), None, None, None, p, None
    q = (r.square().mean(1) + s["eps"]).rsqrt()
    x = r * q.unsqueeze(1) * s["w_pre"]
    out = _quantized(x, s["fmt"]) if s["fmt"] != "none" else (None, None)
    return r.to(s["r"].dtype), *out, x.bfloat16() if s["bf16"] else None, p, q


def _plain_norm_bwd(s):
    d, dw_pre, dw_post, dgate = s["dr"].float(), None, None, None
    if s["pre"]:
        n = s["r"].float() * s["rstd_pre"].unsqueeze(1)
        dx = s["dx"].float()
        dw_pre = (dx * n).sum(0)
        e = dx * s["w_pre"]
        d = d + s["rstd_pre"].unsqueeze(1) * (e - n * (e * n).mean(1, keepdim=True))
    n = s["h"].float()
    if s["post"]:
        n = n * s["rstd_post"].unsqueeze(1)
    e = d * s["res_scale"]
    if s["gate"] is not None:
        sig = 1 / (1 + torch.exp(-s["gate"].float()))
        dgate = (e * n * s["w_post"] * sig * (1 - sig)).bfloat16()
        e = e * sig
    dw_post = (e * n).sum(0)
    e = e * s["w_post"]
    if s["post"]:
        e = s["rstd_post"].unsqueeze(1) * (e - n * (e * n).mean(1, keepdim=True))
    return d.to(s["dr"].dtype), e.bfloat16(), dgate, dw_post, dw_pre


PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "save": _plain_save, "restore": _plain_restore,
         "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    T, op = case["T"], case["op"]
    if op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        item = 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return {"bytes": T * E * item + 8 * T * k + 4 * E + (4 * E if case["bias"] else 0),
                    "flops": T * E * (6 + k)}
        # the sigmoid's gradient needs the chosen logits alone, the softmax's needs all of them
        read = T * E * item if case["scores"] == "softmax" else T * k * item
        return {"bytes": read + 8 * T * k + T * E * item, "flops": 8 * T * E}
    if op in ("save", "restore"):
        H = case["H"]
        row = 4 if case["weighted"] else 0
        if op == "save":
            return {"bytes": T * (4 * H + H + 2 * H + 3 * H // GROUP * 4 + row), "flops": 14 * T * H}
        out = 4 * H if case["fmt"] == "bf16" else 2 * H + 2 * H // GROUP * 4
        return {"bytes": T * (2 * H + 2 * H // GROUP * 4 + 2 * H + out + (2 * H if case["y"] else 0) + 2 * row),
                "flops": 22 * T * H}
    C = case["C"]
    res = 4 if case["residual"] == "f32" else 2
    gate = 2 if case["gate"] else 0
    if op == "norm":
        out = (1 + 4 / GROUP if case["fmt"] != "none" else 0) + (2 if case["bf16"] else 0)
        return {"bytes": int(T * C * (2 + gate + 2 * res + out)) + 8 * T + 8 * C, "flops": 14 * T * C}
    pre = 2 if case["pre"] else 0
    # the stream itself is read for the pre-norm alone
    return {"bytes": T * C * (pre + (res if pre else 0) + res + 2 + gate + res + 2 + gate) + 8 * T + 16 * C,
            "flops": 24 * T * C}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; codes as the unrounded quotients, and None for
    whole numbers.  Rows are independent, so they are taken in pieces; weight gradients are added up."""
    s = prepare(case, seed)
    f = {"route": _exact_route, "route_bwd": _exact_route_bwd, "save": _exact_save, "restore": _exact_restore,
         "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}[case["op"]]
    whole = {"w_post", "w_pre", "bias"}
    parts = []
    for lo in range(0, case["T"], 8192):
        piece = {n: v[lo:lo + 8192] if isinstance(v, torch.Tensor) and n not in whole else v for n, v in s.items()}
        parts.append(f({n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for n, v in piece.items()}))
    if isinstance(parts[0], torch.Tensor):
        return torch.cat(parts)
    joined = []
    for i, v in enumerate(parts[0]):
        if v is None:
            joined.append(None)
        elif case["op"] == "norm_bwd" and i >= 3:  # dw_post, dw_pre
            joined.append(torch.stack([p[i] for p in parts]).sum(0))
        else:
            joined.append(torch.cat([p[i] for p in parts]))
    return tuple(joined)


def _exact_shares(x, kind):
    if kind == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, 1).nan_to_num(0.0)


def _exact_route(s):
    x = s["logits"]
    share = _exact_shares(x, s["scores"])
    key = share.clone() if s["bias"] is None else share + s["bias"]
    key[x == -math.inf] = -math.inf
    G = s["groups"]
    if G > 1:
        best = key.view(len(x), G, -1).sort(2, descending=True).values[:, :, :2]
        total = best.nan_to_num(neginf=0.0).sum(2)
        total[best[:, :, 0] == -math.inf] = -math.inf
        out = total.sort(dim=1, descending=True, stable=True).indices[:, s["topk_groups"]:]
        key.view(len(x), G, -1).scatter_(1, out.unsqueeze(2).expand(-1, -1, key.shape[1] // G), -math.inf)
    order = key.sort(dim=1, descending=True, stable=True)
    w = share.gather(1, order.indices[:, :s["k"]])
    w[order.values[:, :s["k"]] == -math.inf] = 0
    if s["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return None, w * s["scale"], None


def _exact_route_bwd(s):
    x, ids, T = s["logits"], s["ids"].long(), len(s["logits"])
    at = torch.arange(T, device=DEV).unsqueeze(1).expand_as(ids)[ids >= 0], ids[ids >= 0]
    g = torch.zeros_like(x)
    g[at] = s["dweights"][ids >= 0] * s["scale"]
    mask = torch.zeros_like(x)
    mask[at] = 1.0
    share = _exact_shares(x, s["scores"])
    if s["renorm"]:  # of share / sum of the chosen shares
        total = (share * mask).sum(1, keepdim=True)
        g = (mask * (g / total - (g * share).sum(1, keepdim=True) / total.square())).nan_to_num(0.0)
    if s["scores"] == "sigmoid":
        return g * share * torch.sigmoid(-x)
    return share * g - share * (share * g).sum(1, keepdim=True)


def _exact_groups(v, fmt):
    v = v.reshape(len(v), -1, GROUP)
    s = v.abs().amax(2).clamp(min=1e-4) / FP8[fmt][1]
    return (v / s[:, :, None]).flatten(1), s


def _exact_save(s):
    g, u = s["x"].chunk(2, 1)
    y = g * torch.sigmoid(g) * u
    y = y if s["w"] is None else y * s["w"][:, None]
    return _exact_groups(y, s["fmt"]) + _exact_groups(s["x"], s["ckpt_fmt"])


def _exact_restore(s):
    x = s["ckpt"] * s["ckpt_sf"].repeat_interleave(GROUP, 1)
    g, u = x.chunk(2, 1)
    sig, rest = torch.sigmoid(g), torch.sigmoid(-g)
    w = 1.0 if s["w"] is None else s["w"][:, None]
    dg = s["dy"] * w * u * (sig + g * sig * rest)
    du = s["dy"] * w * g * sig
    dw = None if s["w"] is None else (s["dy"] * g * sig * u).sum(1)
    y = w * g * sig * u if s["y"] else None
    dx = torch.cat([dg, du], 1)
    return (dx, None, dw, y) if s["fmt"] == "bf16" else (*_exact_groups(dx, s["fmt"]), dw, y)


def _exact_norm(s):
    C = s["C"]
    p = (s["h"].pow(2).sum(1) / C + s["eps"]).pow(-0.5) if s["post"] else None
    branch = s["w_post"] * s["h"] * (1.0 if p is None else p[:, None])
    if s["gate"] is not None:
        branch = branch * torch.sigmoid(s["gate"])
    r = s["r"] + branch * s["res_scale"]
    if not s["pre"]:
        return r, None, None, None, p, None
    q = (r.pow(2).sum(1) / C + s["eps"]).pow(-0.5)
    x = s["w_pre"] * r * q[:, None]
    codes = (None, None) if s["fmt"] == "none" else _exact_groups(x, s["fmt"])
    return (r, *codes, x if s["bf16"] else None, p, q)


def _exact_norm_bwd(s):
    C, dr, dw_pre, dgate = s["C"], s["dr"], None, None
    if s["pre"]:
        r, q = s["r"], s["rstd_pre"][:, None]
        dw_pre = (s["dx"] * r * q).sum(0)
        inner = (s["dx"] * s["w_pre"] * r).sum(1, keepdim=True)
        dr = dr + q * s["dx"] * s["w_pre"] - r * q.pow(3) * inner / C
    sig = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"])
    p = s["rstd_post"][:, None] if s["post"] else 1.0
    db = s["res_scale"] * dr
    dw_post = (db * sig * s["h"] * p).sum(0)
    if s["gate"] is not None:
        dgate = db * s["w_post"] * s["h"] * p * sig * torch.sigmoid(-s["gate"])
    dh = db * sig * s["w_post"] * p
    if s["post"]:
        dh = dh - s["h"] * p.pow(3) * (db * sig * s["w_post"] * s["h"]).sum(1, keepdim=True) / C
    return dr, dh, dgate, dw_post, dw_pre
