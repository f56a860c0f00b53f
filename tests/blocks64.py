"""The operators around an FP8 block in 64 bits, straight from their formulas
(test infrastructure): expert routing, the SwiGLU from its 8-bit checkpoint and
the norms around a block, each with its gradients.  Inputs and outputs are
float64 torch tensors on the CPU."""
from __future__ import annotations

import torch

INF = float("inf")
LARGEST = float(torch.finfo(torch.float32).max)


# --- routing -----------------------------------------------------------------

def scores(x, kind):
    live = x > -INF                     # false for NaN too
    x = torch.where(live, x.clamp(max=LARGEST), -INF)
    if kind == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top > -INF, top, 0.0))
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total > 0, total, 1.0)
    return torch.where(live, s, 0.0), live


def keys(x, kind, bias):
    s, live = scores(x, kind)
    key = s if bias is None else s + bias
    return s, torch.where(live & (key > -INF), key, -INF)


def route(x, k, kind="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renorm=True,
          scale=1.0):
    """One row at a time, by sorting (key, -index)."""
    s, key = keys(x, kind, bias)
    T, E = x.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    per = E // groups
    for t in range(T):
        row = key[t].tolist()
        if groups > 1:
            of = []
            for g in range(groups):
                have = sorted((v for v in row[g * per:(g + 1) * per] if v > -INF), reverse=True)
                of.append(sum(have[:group_top]) if have else -INF)
            best = sorted(range(groups), key=lambda g: (-of[g], g))[:topk_groups]
            row = [v if e // per in best else -INF for e, v in enumerate(row)]
        order = [e for e in sorted(range(E), key=lambda e: (-row[e], e))[:k] if row[e] > -INF]
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        w[t, :len(order)] = s[t, order]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def route_weights(x, ids, kind, renorm, scale):
    """The weights of given ids, as a function of the logits."""
    s, _ = scores(x, kind)
    ok = (ids >= 0) & (ids < x.shape[1])
    p = torch.where(ok, s.gather(1, torch.where(ok, ids, 0).long()), 0.0)
    if renorm:
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return p * scale


def route_backward(x, ids, dw, kind, renorm, scale):
    s, live = scores(x, kind)
    ok = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(ok, ids, 0).long()
    p = torch.where(ok, s.gather(1, at), 0.0)
    a = torch.where(ok, dw * scale, 0.0)
    if renorm:
        total = p.sum(1, keepdim=True)
        safe = torch.where(total > 0, total, 1.0)
        a = torch.where(ok & (total > 0), (a - (a * p).sum(1, keepdim=True) / safe) / safe, 0.0)
    ds = torch.zeros_like(x).scatter_add_(1, at, torch.where(ok, a, 0.0))
    if kind == "sigmoid":
        dx = ds * s * torch.sigmoid(torch.where(live, -x, 0.0))
    else:
        dx = s * (ds - (ds * s).sum(1, keepdim=True))
    return torch.where(live, dx, 0.0)


# --- SwiGLU ------------------------------------------------------------------

def swiglu(x, w=None):
    g, u = x.chunk(2, 1)
    y = g * torch.sigmoid(g) * u
    return y if w is None else y * w[:, None]


def swiglu_backward(x, dy, w=None):
    """dx, the gradient of w."""
    g, u = x.chunk(2, 1)
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    wt = 1.0 if w is None else w[:, None]
    return (torch.cat([dy * u * s * (1 + g * rest) * wt, dy * g * s * wt], 1),
            (dy * g * s * u).sum(1))


# --- norms -------------------------------------------------------------------

def residual_norm(r, h=None, w_post=None, gate=None, w_pre=None, post=True, a=1.0, eps=1e-6,
                  pre=True):
    """r', x, p, q."""
    p = q = x = None
    if h is not None:
        b = h
        if post:
            p = (h.square().mean(1) + eps) ** -0.5
            b = b * p[:, None]
        if w_post is not None:
            b = b * w_post
        if gate is not None:
            b = b * torch.sigmoid(gate)
        r = r + a * b
    if pre:
        q = (r.square().mean(1) + eps) ** -0.5
        x = r * q[:, None]
        if w_pre is not None:
            x = x * w_pre
    return r, x, p, q


def residual_norm_backward(dr, r, h=None, dx=None, w_post=None, gate=None, w_pre=None, p=None,
                           q=None, a=1.0):
    """dr of the input stream, dh, dgate, dw_post, dw_pre; r is the forward's r'."""
    dh = dgate = dw_post = dw_pre = None
    dr = torch.zeros_like(dx) if dr is None else dr
    if dx is not None:
        n = r * q[:, None]
        e = dx if w_pre is None else dx * w_pre
        dw_pre = (dx * n).sum(0)
        dr = dr + q[:, None] * (e - n * (e * n).mean(1, keepdim=True))
    if h is not None:
        m = h if p is None else h * p[:, None]
        s = torch.ones_like(h) if gate is None else torch.sigmoid(gate)
        wp = torch.ones(h.shape[1], dtype=h.dtype) if w_post is None else w_post
        e = a * dr
        if gate is not None:
            dgate = e * m * wp * s * (1 - s)
        dw_post = (e * s * m).sum(0)
        f = e * s * wp
        dh = f if p is None else p[:, None] * (f - m * (f * m).mean(1, keepdim=True))
    return dr, dh, dgate, dw_post, dw_pre
