"""The formulas of the experts' operators in 64 bits, on the CPU, as plainly as they can be written:
what tests compare the kernels with."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 128


def order(ids, experts, align, rows):
    """slots, rows and offsets of routed pairs, by walking the experts in turn."""
    flat = ids.flatten().tolist()
    slots, of_row, offsets, at = [-1] * len(flat), [-1] * rows, [0], 0
    for e in range(experts):
        for p, x in enumerate(flat):
            if x == e:
                slots[p], of_row[at] = at, p
                at += 1
        at = -(-at // align) * align
        offsets.append(at)
    i32 = torch.int32
    return (torch.tensor(slots, dtype=i32).view(ids.shape), torch.tensor(of_row, dtype=i32),
            torch.tensor(offsets, dtype=i32))


def reduce(y, slots, weights=None):
    """(out, sum of magnitudes) in 64 bits."""
    y = torch.cat([y.double(), torch.zeros(1, y.shape[1], dtype=torch.float64)])
    at = torch.where((slots >= 0) & (slots < len(y) - 1), slots, len(y) - 1).long()
    terms = y[at]
    if weights is not None:
        terms = terms * weights.double().unsqueeze(2)
        terms[at == len(y) - 1] = 0
    return terms.sum(1), terms.abs().sum(1)


def reduce_backward(dout, y, slots, weights):
    """(dy of the pairs [T, k, C], dweights, magnitudes of dweights)."""
    live = (slots >= 0) & (slots < len(y))
    at = torch.where(live, slots, 0).long()
    d = dout.double().unsqueeze(1)
    terms = torch.where(live.unsqueeze(2), d * y.double()[at], 0.0)
    return weights.double().unsqueeze(2) * d, terms.sum(2), terms.abs().sum(2)


def spread(pairs, slots, rows, fill=0.0):
    """Pairs [T, k, ...] at their rows [rows, ...], `fill` elsewhere."""
    out = torch.full((rows, *pairs.shape[2:]), fill, dtype=pairs.dtype)
    live = (slots >= 0) & (slots < rows)
    out[slots[live].long()] = pairs[live]
    return out


def decoded(codes, sf):
    """Codes [..., C] times scales [..., C/128]."""
    return codes.double() * sf.double().repeat_interleave(GROUP, -1)


def product(a, a_sf, w, w_sf, offsets):
    """(out [R, N], magnitudes), zeros for the rows of no expert."""
    x = decoded(a, a_sf)
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        m = w[e].double() * w_sf[e].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        out[lo:hi] = x[lo:hi] @ m.T
        size[lo:hi] = x[lo:hi].abs() @ m.abs().T
    return out, size


def weight_grad(dy_t, dy_sf, x_t, x_sf, offsets):
    """(dw [E, N, K], magnitudes)."""
    dy, x = decoded(dy_t, dy_sf), decoded(x_t, x_sf)
    spans = list(zip(offsets.tolist(), offsets.tolist()[1:]))
    return (torch.stack([dy[:, lo:hi] @ x[:, lo:hi].T for lo, hi in spans]),
            torch.stack([dy[:, lo:hi].abs() @ x[:, lo:hi].abs().T for lo, hi in spans]))


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def w4_decoded(codes, sf):
    """4-bit codes [..., K/2] (the low nibble is the even column) times their scales: UE8M0 bytes
    (uint8) or fp32."""
    c = codes.numpy()
    v = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(*c.shape[:-1], -1)
    s = np.exp2(sf.numpy().astype(np.float64) - 127) if sf.dtype == torch.uint8 else sf.double().numpy()
    return torch.from_numpy(v * np.repeat(s, v.shape[-1] // s.shape[-1], -1))


def w4_product(x, x_sf, w, w_sf, ids, each):
    """(out [T k, N], magnitudes): zeros for empty slots."""
    rows = decoded(x, x_sf)
    m = w4_decoded(w, w_sf)
    if ids is None:
        return rows @ m.T, rows.abs() @ m.abs().T
    T, k = ids.shape
    rows = rows if each else rows.repeat_interleave(k, 0)
    out = torch.zeros(T * k, m.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for p, e in enumerate(ids.flatten().tolist()):
        if 0 <= e < m.shape[0]:
            out[p], size[p] = m[e] @ rows[p], m[e].abs() @ rows[p].abs()
    return out, size
