"""What the experts of a mixture are measured on, from routing to their outputs: tokens sorted by expert
and back with their weights, in both directions; the experts' products of FP8 codes and scales, with the
weight gradient; and products of few tokens with 4-bit weights.

``own`` False computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end); ``own`` True makes the calls a user makes of this package.  FP8 outputs are returned as
float8 tensors, which hold the values their codes stand for, beside their fp32 scales.  Where an output
has rows behind the last expert's, which a call leaves as they were, it goes to a zeroed buffer that the
program keeps.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = 128
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # a decoding step of 4 sequences: each token to 8 of 256 experts, cast on the way; latency counts
        dict(name="sort, 4 tokens", op="sort", T=4, k=8, E=256, C=7168, align=1, form="cast", fmt="e4m3",
             weighted=True, dropped=False),
        # a training batch of 8192 tokens to 8 of 64 experts, groups of 128 rows for the transposed casts
        dict(name="sort, 8192 tokens", op="sort", T=8192, k=8, E=64, C=4096, align=128, form="cast",
             fmt="e4m3", weighted=True, dropped=False),
        # the gradient of sorting an odd batch, with tokens that have empty slots, and the gradients of
        # the rows' weights
        dict(name="back, 1021 tokens", op="back", T=1021, k=6, E=60, C=1408, align=128, weighted=False,
             values=True, dropped=True, out="bf16"),
        # the experts' outputs of the training batch, weighted and summed for each token
        dict(name="back, 8192 tokens", op="back", T=8192, k=8, E=64, C=4096, align=128, weighted=True,
             values=False, dropped=False, out="bf16"),
        # the backward of a weighted sum on a small odd batch, gradients cast for the next product
        dict(name="back backward, 333 tokens", op="back_bwd", T=333, k=4, E=12, C=640, align=128,
             form="cast", fmt="e5m2", dropped=True),
        # the same on the training batch: bf16 gradients and those of the weights
        dict(name="back backward, 8192 tokens", op="back_bwd", T=8192, k=8, E=64, C=4096, align=128,
             form="bf16", fmt="e4m3", dropped=False),
        # a short prompt: a few rows for each of 60 experts, where reading the weights counts
        dict(name="product, 384 rows", op="product", rows=384, E=60, N=2816, K=2048, align=1, fmt="e4m3"),
        # the first product of the training batch's experts (gate and up of H = 2048), 32 experts
        dict(name="product, 65536 rows", op="product", rows=65536, E=32, N=4096, K=4096, align=128,
             fmt="e4m3"),
        # the weight gradient of a small ragged batch, experts without rows among them
        dict(name="weight gradient, 1100 rows", op="weight_grad", rows=1100, E=12, N=768, K=640,
             fmt="e5m2", out="f32"),
        # the weight gradient of the first product, 65536 rows of 8 experts
        dict(name="weight gradient, 65536 rows", op="weight_grad", rows=65536, E=8, N=4096, K=4096,
             fmt="e4m3", out="f32"),
        # one token at a time: the first product of its 8 of 64 experts with 4-bit weights
        dict(name="4-bit product, 1 token", op="w4", T=1, k=8, E=64, N=4096, K=4096, group=32, each=False),
        # 48 sequences decoded together: the second product, each expert's rows with their own input
        dict(name="4-bit product, 48 tokens", op="w4", T=48, k=8, E=64, N=4096, K=2048, group=32, each=True),
    ]


def draw(rng):
    def size(lo, hi):
        n = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))
        return n + 1 if n == 3072 else n

    def width(most):
        n = size(1, most)
        return GROUP * (n + 1 if n in (12, 24) else n)

    op = rng.choice(["sort", "back", "back_bwd", "product", "weight_grad", "w4"])
    if op in ("sort", "back", "back_bwd"):
        c = dict(op=op, k=rng.randint(1, 8), C=width(56), align=rng.choice([1, 16, 128]),
                 dropped=rng.random() < 0.4)
        c["E"] = max(c["k"], size(2, 256))
        c["T"] = size(1, min(16384, 8192 * 8 * 4096 // (c["k"] * c["C"])))
        c["dropped"] = c["dropped"] and c["T"] >= 8  # at least one token has a slot
        if op == "sort":
            c.update(form=rng.choice(["cast", "cast", "codes", "bf16"]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                     weighted=rng.random() < 0.7)
            c["T"] = max(1, c["T"] // 2) if c["form"] == "bf16" else c["T"]
        elif op == "back":
            c.update(weighted=rng.random() < 0.6, values=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
        else:
            c.update(form=rng.choice(["cast", "bf16"]), fmt=rng.choice(["e4m3", "e5m2"]))
    elif op == "product":
        c = dict(op=op, E=size(1, 64), N=width(32), K=width(32), align=rng.choice([1, 16, 128]),
                 fmt=rng.choice(["e4m3", "e4m3", "e5m2"]))
        c["rows"] = size(1, 32768)
    elif op == "weight_grad":
        c = dict(op=op, E=size(1, 16), N=width(32), K=width(32), fmt=rng.choice(["e4m3", "e5m2"]),
                 out=rng.choice(["f32", "bf16"]))
        c["rows"] = size(1, 32768)
    else:
        c = dict(op=op, N=width(32), K=width(32), group=rng.choice([32, 32, 128]), T=size(1, 64))
        c["k"] = rng.choice([0, 1, 2, 4, 8])  # 0: one matrix for all tokens
        c["E"] = max(c["k"], size(1, 64)) if c["k"] else 1
        c["each"] = c["k"] > 0 and rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _capacity(P, E, align):
    return (P + min(E, P) * (align - 1)) // align * align


def _ids(gen, T, k, E, dropped):
    """k different experts of each token, some experts liked better than others; with ``dropped`` some
    slots empty and every 16th token without any."""
    liking = torch.randn(E, generator=gen, device=DEV)
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_min(1e-20)
    ids = (liking - torch.log(-torch.log(u))).topk(k, 1).indices.int()
    if dropped:
        ids = torch.where(torch.rand(T, k, generator=gen, device=DEV) < 0.1, -1, ids)
        ids[::16] = -1
    return ids.contiguous()


def _quantized(x, fmt):
    """Codes and scales of 1x128 groups of an fp32 matrix."""
    dtype, top = FP8[fmt]
    v = x.view(x.shape[0], -1, GROUP)
    s = v.abs().amax(2).clamp_min(1e-4) / top
    return (v / s.unsqueeze(2)).view_as(x).to(dtype), s


def _offsets(gen, rows, E, align):
    """Starts of the experts' rows: uneven shares, some of none; multiples of ``align``."""
    share = torch.rand(E, generator=gen, device=DEV) ** 2 + 1e-3
    share[torch.rand(E, generator=gen, device=DEV) < 0.1] = 0.0
    share = (share / share.sum().clamp_min(1e-9)).tolist()
    sizes, left = [], rows
    for e in range(E):
        n = min(left, round(rows * share[e]))
        sizes.append(n)
        left -= n
    sizes[-1] += left
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (n + align - 1) // align * align)
    return torch.tensor(starts, dtype=torch.int32, device=DEV), starts


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    op, s = case["op"], dict(case)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    def codes(rows, cols, fmt, std=1.0):
        """FP8 codes and scales of a normal matrix, made in pieces."""
        parts = [_quantized(normal(min(16384, rows - lo), cols, std=std, dtype=torch.float32), fmt)
                 for lo in range(0, rows, 16384)]
        return (torch.cat([p[0].view(torch.uint8) for p in parts]).view(FP8[fmt][0]),
                torch.cat([p[1] for p in parts]))

    if op in ("sort", "back", "back_bwd"):
        T, k, E, C = case["T"], case["k"], case["E"], case["C"]
        s["ids"] = _ids(gen, T, k, E, case["dropped"])
        s["R"] = R = _capacity(T * k, E, case["align"])
        w = torch.rand(T, k, generator=gen, device=DEV) + 0.01
        s["w"] = w / w.sum(1, keepdim=True) if op == "back_bwd" or case["weighted"] else None
        form = case.get("form")
        if op == "sort":
            if form == "codes":
                s["x"], s["x_sf"] = codes(T, C, case["fmt"])
            else:
                s["x"], s["x_sf"] = normal(T, C), None
        else:
            # what the forward pass left behind
            s["slots"], s["rows"], s["offsets"] = _plain_order(s["ids"], E, case["align"], R)
            if op == "back":
                s["y"] = normal(R, C)
                s["row_values"] = normal(R, dtype=torch.float32) if case["values"] else None
            else:
                s["y"], s["dout"] = normal(R, C), normal(T, C, std=0.5)
        if op != "back":
            if form == "bf16":
                s["out"], s["out_sf"] = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV), None
            else:
                s["out"] = torch.zeros(R, C, dtype=torch.uint8, device=DEV).view(FP8[case["fmt"]][0])
                s["out_sf"] = torch.zeros(R, C // GROUP, device=DEV)
            s["row_w"] = torch.zeros(R, device=DEV) if op == "sort" and case["weighted"] else None
        if own and op != "sort":
            import fp8_activation_quantization_gb300 as tkq
            s["order"] = tkq.ExpertOrder(s["slots"], s["rows"], s["offsets"])
    elif op == "product":
        E, N, K = case["E"], case["N"], case["K"]
        s["offsets"], s["starts"] = _offsets(gen, case["rows"], E, case["align"])
        # rows behind the last expert's stay as they are
        R = _capacity(case["rows"], E, case["align"]) + 5
        s["a"], s["a_sf"] = codes(R, K, case["fmt"])
        w = normal(E * N, K // GROUP, GROUP, std=K ** -0.5)
        block = w.float().abs().amax(2).view(E, N // GROUP, GROUP, K // GROUP).amax(2).clamp_min(1e-4) / 448.0
        s["w"] = torch.cat([(w[e * N:(e + 1) * N] / block[e].repeat_interleave(GROUP, 0).unsqueeze(2))
                            .to(torch.float8_e4m3fn).view(torch.uint8) for e in range(E)]) \
            .view(E, N, K).view(torch.float8_e4m3fn)
        s["w_sf"] = block
        s["out"] = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    elif op == "weight_grad":
        E, N, K = case["E"], case["N"], case["K"]
        s["offsets"], s["starts"] = _offsets(gen, case["rows"], E, GROUP)
        R = _capacity(case["rows"], E, GROUP)  # the rows in use and some behind them
        s["dy"], s["dy_sf"] = codes(N, R, case["fmt"], std=0.5)
        s["x"], s["x_sf"] = codes(K, R, "e4m3")
    else:
        T, k, E, N, K = (case[n] for n in "TkENK")
        s["ids"] = _ids(gen, T, k, E, False) if k else None
        s["x"], s["x_sf"] = codes(T * k if case["each"] else T, K, "e4m3")
        shape = (E, N) if k else (N,)
        s["w4"] = torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, generator=gen, device=DEV)
        size = torch.rand(*shape, K // case["group"], generator=gen, device=DEV) + 0.5
        if case["group"] == 32:  # UE8M0: exponents of powers of two
            s["w4_sf"] = torch.randint(117, 122, size.shape, dtype=torch.uint8, generator=gen, device=DEV)
        else:
            s["w4_sf"] = size * K ** -0.5 / 3
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


def _own(s):
    import fp8_activation_quantization_gb300 as tkq
    op = s["op"]
    if op == "sort":
        order = tkq.expert_order(s["ids"], s["E"], align=s["align"])
        out, sf, row_w = tkq.expert_gather(s["x"], order, fmt=s["fmt"] if s["form"] == "cast" else None,
                                           x_sf=s["x_sf"], weights=s["w"], out=s["out"], out_sf=s["out_sf"],
                                           row_weights=s["row_w"])
        return order.slots, order.rows, order.offsets, out, sf, row_w
    if op == "back":
        return tkq.expert_reduce(s["y"], s["order"], weights=s["w"], row_values=s["row_values"],
                                 out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    if op == "back_bwd":
        return tkq.expert_reduce_backward(s["dout"], s["y"], s["order"], weights=s["w"],
                                          fmt=s["fmt"] if s["form"] == "cast" else None, out=s["out"],
                                          out_sf=s["out_sf"])
    if op == "product":
        return tkq.expert_product(s["a"], s["a_sf"], s["w"], s["w_sf"], s["offsets"], out=s["out"])
    if op == "weight_grad":
        return tkq.expert_weight_grad(s["dy"], s["dy_sf"], s["x"], s["x_sf"], s["offsets"],
                                      out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    return tkq.w4_product(s["x"], s["x_sf"], s["w4"], s["w4_sf"], ids=s["ids"])


def _plain_order(ids, E, align, R):
    flat = ids.flatten()
    P = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E).long()
    perm = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.cat([torch.zeros_like(padded[:1]), padded.cumsum(0)])
    before = counts.cumsum(0) - counts  # pairs of smaller experts
    rank = torch.arange(P, device=DEV) - before[key[perm]]
    taken = key[perm] < E
    slot = torch.where(taken, offsets[key[perm]] + rank, R)
    slots = torch.empty_like(flat).index_copy_(0, perm, torch.where(taken, slot, -1).int())
    rows = torch.full((R + 1,), -1, dtype=torch.int32, device=DEV)
    rows[slot] = torch.where(taken, perm, -1).int()
    return slots.view(ids.shape), rows[:R].contiguous(), offsets.int()


def _plain_spread(v, slots, R):
    """Rows v [T, k, ...] or [T, 1, ...] to their slots, zeros elsewhere."""
    T, k = slots.shape
    at = torch.where(slots >= 0, slots, R).long().flatten()
    out = torch.zeros(R + 1, *v.shape[2:], dtype=v.dtype, device=DEV)
    for j in range(k):
        out[at.view(T, k)[:, j]] = v[:, min(j, v.shape[1] - 1)]
    return out[:R]


def _as_bytes(v):
    return v.view(torch.uint8)


def _plain_sort(s):
    slots, rows, offsets = _plain_order(s["ids"], s["E"], s["align"], s["R"])
    x, sf = s["x"], s["x_sf"]
    if s["form"] == "cast":
        x, sf = _quantized(x.float(), s["fmt"])
    if sf is None:
        out = _plain_spread(x.unsqueeze(1), slots, s["R"])
    else:
        out = _plain_spread(_as_bytes(x).unsqueeze(1), slots, s["R"]).view(x.dtype)
        sf = _plain_spread(sf.unsqueeze(1), slots, s["R"])
        if s["form"] == "cast":  # padding rows are zeros, cast like any other
            pad = (rows < 0) & (torch.arange(s["R"], device=DEV) < offsets[-1])
            sf = torch.where(pad.unsqueeze(1), torch.full_like(sf, 1e-4) / FP8[s["fmt"]][1], sf)
    row_w = _plain_spread(s["w"], slots, s["R"]) if s["w"] is not None else None
    return slots, rows, offsets, out, sf, row_w


def _plain_back(s):
    slots = s["slots"]
    T, k = slots.shape
    at, there = slots.clamp_min(0).long(), slots >= 0
    out = torch.zeros(T, s["C"], device=DEV)
    for j in range(k):
        v = s["y"][at[:, j]].float()
        if s["w"] is not None:
            v = v * s["w"][:, j:j + 1]
        out += torch.where(there[:, j:j + 1], v, 0)
    values = None
    if s["row_values"] is not None:
        values = torch.where(there, s["row_values"][at], 0)
    return out.to(torch.bfloat16) if s["out"] == "bf16" else out, values


def _plain_back_bwd(s):
    slots, R, C = s["slots"], s["R"], s["C"]
    T, k = slots.shape
    d = s["dout"].float()
    at, there = slots.clamp_min(0).long(), slots >= 0
    dw = torch.stack([(d * s["y"][at[:, j]].float()).sum(1) for j in range(k)], 1)
    dw = torch.where(there, dw, 0)
    # a weight times a row, slot by slot
    spread = torch.zeros(R + 1, C, device=DEV)
    for j in range(k):
        spread[torch.where(there[:, j], slots[:, j], R).long()] = d * s["w"][:, j:j + 1]
    dy = spread[:R]
    if s["form"] == "bf16":
        return dy.bfloat16(), None, dw
    codes, sf = _quantized(dy, s["fmt"])
    return codes, torch.where((torch.arange(R, device=DEV) < s["offsets"][-1]).unsqueeze(1), sf, 0), dw


def _plain_product(s):
    starts, N, K = s["starts"], s["N"], s["K"]
    out = torch.zeros(s["a"].shape[0], N, dtype=torch.bfloat16, device=DEV)
    for e in range(s["E"]):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        a = (s["a"][lo:hi].float().view(hi - lo, -1, GROUP) * s["a_sf"][lo:hi].unsqueeze(2)).view(hi - lo, K)
        w = s["w"][e].float().view(N // GROUP, GROUP, K // GROUP, GROUP) * s["w_sf"][e][:, None, :, None]
        out[lo:hi] = (a @ w.view(N, K).t()).bfloat16()
    return out


def _plain_weight_grad(s):
    starts, N, K = s["starts"], s["N"], s["K"]
    out = torch.zeros(s["E"], N, K, dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32, device=DEV)
    for e in range(s["E"]):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        g = slice(lo // GROUP, hi // GROUP)
        dy = (s["dy"][:, lo:hi].float().view(N, -1, GROUP) * s["dy_sf"][:, g].unsqueeze(2)).view(N, -1)
        x = (s["x"][:, lo:hi].float().view(K, -1, GROUP) * s["x_sf"][:, g].unsqueeze(2)).view(K, -1)
        out[e] = dy @ x.t()
    return out


def _plain_w4(s):
    x = (s["x"].float().view(-1, s["K"] // GROUP, GROUP) * s["x_sf"].unsqueeze(2)).view(-1, s["K"])
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    sf = s["w4_sf"]
    sf = torch.exp2(sf.float() - 127) if s["group"] == 32 else sf

    def matrix(codes, scales):
        both = torch.stack([codes & 15, codes >> 4], -1).long()  # the low nibble is the even column
        return (table[both].view(s["N"], -1, s["group"]) * scales.unsqueeze(2)).view(s["N"], s["K"])

    if s["ids"] is None:
        return (x @ matrix(s["w4"], sf).t()).bfloat16()
    T, k = s["ids"].shape
    rows = x if s["each"] else x.repeat_interleave(k, 0)
    flat = s["ids"].flatten()
    out = torch.zeros(T * k, s["N"], dtype=torch.bfloat16, device=DEV)
    for e in flat.unique().tolist():
        at = (flat == e).nonzero().flatten()
        out[at] = (rows[at] @ matrix(s["w4"][e], sf[e]).t()).bfloat16()
    return out


PLAIN = {"sort": _plain_sort, "back": _plain_back, "back_bwd": _plain_back_bwd, "product": _plain_product,
         "weight_grad": _plain_weight_grad, "w4": _plain_w4}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("sort", "back", "back_bwd"):
        T, k, E, C = case["T"], case["k"], case["E"], case["C"]
        P = T * k
        live = P * 0.84 if case["dropped"] else P  # slots in use
        if op == "sort":
            scales = C // GROUP * 4
            read = {"cast": 2 * C, "bf16": 2 * C, "codes": C + scales}[case["form"]]
            write = 2 * C if case["form"] == "bf16" else C + scales
            order = 8 * P + 4 * _capacity(P, E, case["align"]) + 4 * E
            return {"bytes": int(T * read + live * write) + order + (8 * P if case["weighted"] else 0),
                    "flops": 4 * T * C if case["form"] == "cast" else T}
        if op == "back":
            item = 2 if case["out"] == "bf16" else 4
            return {"bytes": int(live * 2 * C) + T * C * item + 4 * P + (4 * P if case["weighted"] else 0)
                    + (8 * P if case["values"] else 0), "flops": int(2 * live * C)}
        write = 2 * C if case["form"] == "bf16" else C + C // GROUP * 4
        return {"bytes": int(2 * T * C + live * (2 * C + write)) + 12 * P, "flops": int(4 * live * C)}
    if op == "product":
        E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
        used = min(E, rows)  # experts that can have rows at all
        return {"bytes": rows * (K + K // 32) + used * (N * K + N * K // GROUP ** 2 * 4) + 2 * rows * N,
                "flops": 2 * rows * N * K}
    if op == "weight_grad":
        E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
        return {"bytes": rows * (N + K) + rows * (N + K) // 32 + E * N * K * (4 if case["out"] == "f32" else 2),
                "flops": 2 * rows * N * K}
    T, k, E, N, K = (case[n] for n in "TkENK")
    # experts of which some token thinks, if all were liked alike
    active = E * (1 - (1 - k / E) ** T) if k else 1
    scales = N * K // 32 if case["group"] == 32 else N * K // 32  # 1 byte of 32, 4 bytes of 128
    M = T * max(k, 1)
    x = (M if case["each"] else T) * (K + K // 32)
    return {"bytes": int(active * (N * K // 2 + scales)) + x + 2 * M * N + 4 * T * k, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, codes too: the quotient's nearest; None for whole
    numbers."""
    s = prepare(case, seed)
    return {"sort": _exact_sort, "back": _exact_back, "back_bwd": _exact_back_bwd, "product": _exact_product,
            "weight_grad": _exact_weight_grad, "w4": _exact_w4}[case["op"]](s)


def _exact_places(s):
    """(pair, row) of every pair that has a row: experts in turn, their pairs in rising order."""
    ids = s["ids"].flatten().tolist()
    lists = [[] for _ in range(s["E"])]
    for p, e in enumerate(ids):
        if e >= 0:
            lists[e].append(p)
    pairs, places, at = [], [], 0
    for mine in lists:
        pairs += mine
        places += range(at, at + len(mine))
        at += -(-len(mine) // s["align"]) * s["align"]
    as_index = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)
    return as_index(pairs), as_index(places), at


def _exact_cast(v, fmt):
    g = v.unflatten(1, (-1, GROUP))
    s = g.abs().amax(-1).clamp(min=1e-4) / FP8[fmt][1]
    q = (g / s[..., None]).flatten(1)
    # the nearest code, ties to even: multiples of a step that is that of the quotient's power of two, and
    # below the smallest normal number that of the subnormals
    digits, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    step = torch.exp2(torch.frexp(q).exponent.sub(1).clamp(min=lowest).double() - digits)
    return ((q / step).round() * step).clamp(-FP8[fmt][1], FP8[fmt][1]), s


def _exact_sort(s):
    pair, place, end = _exact_places(s)
    R, C, k = s["R"], s["C"], s["k"]
    x = s["x"].double()
    if s["form"] == "bf16":
        out = torch.zeros(R, C, dtype=torch.float64, device=DEV)
        out[place] = x[pair // k]
        sf = None
    else:
        codes, scale = (x, s["x_sf"].double()) if s["form"] == "codes" else _exact_cast(x, s["fmt"])
        out = torch.zeros(R, C, dtype=torch.float64, device=DEV)
        sf = torch.zeros(R, C // GROUP, dtype=torch.float64, device=DEV)
        if s["form"] == "cast":
            sf[:end] = 1e-4 / FP8[s["fmt"]][1]
        out[place], sf[place] = codes[pair // k], scale[pair // k]
    row_w = None
    if s["w"] is not None:
        row_w = torch.zeros(R, dtype=torch.float64, device=DEV)
        row_w[place] = s["w"].double().flatten()[pair]
    return None, None, None, out, sf, row_w


def _exact_back(s):
    pair, place, _ = _exact_places(s)
    T, k, C = s["T"], s["k"], s["C"]
    out = torch.zeros(T, C, dtype=torch.float64, device=DEV)
    for lo in range(0, len(pair), 16384):
        p, r = pair[lo:lo + 16384], place[lo:lo + 16384]
        v = s["y"][r].double()
        out.index_add_(0, p // k, v if s["w"] is None else v * s["w"].flatten()[p].double()[:, None])
    values = None
    if s["row_values"] is not None:
        values = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        values[pair] = s["row_values"].double()[place]
        values = values.view(T, k)
    return out, values


def _exact_back_bwd(s):
    pair, place, end = _exact_places(s)
    T, k, C = s["T"], s["k"], s["C"]
    dy = torch.zeros(s["R"], C, dtype=torch.float64, device=DEV)
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    for lo in range(0, len(pair), 16384):
        p, r = pair[lo:lo + 16384], place[lo:lo + 16384]
        d = s["dout"][p // k].double()
        dy[r] = s["w"].flatten()[p].double()[:, None] * d
        dw[p] = (s["y"][r].double() * d).sum(1)
    if s["form"] == "bf16":
        return dy, None, dw.view(T, k)
    codes, sf = _exact_cast(dy, s["fmt"])
    sf[end:] = 0
    return codes, sf, dw.view(T, k)


def _exact_product(s):
    out = torch.zeros(s["a"].shape[0], s["N"], dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(zip(s["starts"], s["starts"][1:])):
        a = s["a"][lo:hi].double() * s["a_sf"][lo:hi].double().repeat_interleave(GROUP, 1)
        scales = s["w_sf"][e].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        out[lo:hi] = torch.einsum("rk,nk->rn", a, s["w"][e].double() * scales)
    return out


def _exact_weight_grad(s):
    dy = s["dy"].double() * s["dy_sf"].double().repeat_interleave(GROUP, 1)
    x = s["x"].double() * s["x_sf"].double().repeat_interleave(GROUP, 1)
    return torch.stack([torch.einsum("nr,kr->nk", dy[:, lo:hi], x[:, lo:hi])
                        for lo, hi in zip(s["starts"], s["starts"][1:])])


def _exact_w4(s):
    group, k = s["group"], s["k"]
    w4 = s["w4"] if k else s["w4"][None]
    sf = s["w4_sf"] if k else s["w4_sf"][None]
    x = s["x"].double() * s["x_sf"].double().repeat_interleave(GROUP, 1)
    M = s["T"] * max(k, 1)
    out = torch.zeros(M, s["N"], dtype=torch.float64, device=DEV)
    of_row = s["ids"].flatten().tolist() if k else [0] * M
    for e in sorted(set(of_row)):
        nibble = torch.empty(s["N"], s["K"], dtype=torch.int32, device=DEV)
        nibble[:, 0::2], nibble[:, 1::2] = (w4[e] % 16).int(), (w4[e] // 16).int()
        exponent, mantissa = nibble // 2 % 4, nibble % 2
        size = torch.where(exponent > 0, (1 + mantissa / 2).double() * 2.0 ** (exponent - 1).double(), mantissa.double() / 2)
        scale = 2.0 ** (sf[e].double() - 127) if group == 32 else sf[e].double()
        w = size * (1.0 - 2.0 * (nibble // 8)) * scale.repeat_interleave(group, 1)
        at = torch.tensor([r for r in range(M) if of_row[r] == e], device=DEV)
        out[at] = x[at if s["each"] or not k else at // k] @ w.t()
    return out
