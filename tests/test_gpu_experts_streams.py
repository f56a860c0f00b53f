"""The experts' operators read their inputs on the current stream: on a side stream each input holds other valid data
until a copy that a long fill delays, and the call comes behind the copy.  A call on any other stream would read the
data from before, whose results are different ones."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
T, C, E, K, N = 200, 384, 7, 3, 256


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def bits(t):
    return t.contiguous().view(torch.uint8)


def inputs(seed):
    """Every input of every call, of the same shapes whatever the seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
    d = dict(ids=torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices.int())
    d["ids"][seed % 5::5, 1] = -1
    d["slots"], d["rows"], d["offsets"] = tkq.expert_order(d["ids"], E)
    R = d["rows"].numel()
    d["x"], d["y"], d["w"] = normal(T, C).bfloat16(), normal(R, C).bfloat16(), torch.rand(T, K, generator=g, device="cuda")
    d["xq"], d["xs"] = tkq.per_token_cast(d["x"])
    d["v"] = normal(R)
    d["a"], d["a_sf"] = tkq.per_token_cast(normal(R, C).bfloat16())
    parts = [tkq.per_block_cast(normal(N, C).bfloat16()) for _ in range(E)]
    d["m"], d["m_sf"] = torch.stack([bits(p[0]) for p in parts]).view(F8), torch.stack([p[1] for p in parts])
    d["t1"], d["t1_sf"] = tkq.per_channel_cast(normal(R, N).bfloat16(), transpose=True)
    d["t2"], d["t2_sf"] = tkq.per_channel_cast(normal(R, C).bfloat16(), transpose=True)
    d["m4"] = normal(E, N, C).bfloat16()
    for group in (32, 128):
        d[f"q{group}"], d[f"q{group}_sf"] = tkq.w4_cast(d["m4"], group)
    return d


def calls(d):
    """(name, call that returns what it wrote); rows that a call leaves as they were are zeros."""
    order = tkq.ExpertOrder(d["slots"], d["rows"], d["offsets"])
    R = d["rows"].numel()
    zero = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")
    sf = lambda: zero(R, C // 128, dtype=F32)
    few, few_sf = d["xq"][:20], d["xs"][:20]
    return [
        ("order", lambda: tkq.expert_order(d["ids"], E)),
        ("gather", lambda: tkq.expert_gather(d["x"], order, weights=d["w"], out=zero(R, C, dtype=BF16),
                                             row_weights=zero(R, dtype=F32))),
        ("gather cast", lambda: tkq.expert_gather(d["x"], order, "e5m2", out=zero(R, C), out_sf=sf())),
        ("gather codes", lambda: tkq.expert_gather(d["xq"], order, x_sf=d["xs"], out=zero(R, C), out_sf=sf())),
        ("reduce", lambda: tkq.expert_reduce(d["y"], order, d["w"], d["v"])),
        ("reduce fp32", lambda: tkq.expert_reduce(d["y"], order, out_dtype=F32)),
        ("reduce backward", lambda: tkq.expert_reduce_backward(d["x"], d["y"], order, d["w"], out=zero(R, C, dtype=BF16))),
        ("reduce backward cast", lambda: tkq.expert_reduce_backward(d["x"], d["y"], order, d["w"], "e4m3", out=zero(R, C),
                                                                    out_sf=sf())),
        ("product", lambda: (tkq.expert_product(d["a"], d["a_sf"], d["m"], d["m_sf"], d["offsets"], out=zero(R, N, dtype=BF16)),)),
        ("weight grad", lambda: (tkq.expert_weight_grad(d["t1"], d["t1_sf"], d["t2"], d["t2_sf"], d["offsets"]),)),
        ("weight grad bf16", lambda: (tkq.expert_weight_grad(d["t1"], d["t1_sf"], d["t2"], d["t2_sf"], d["offsets"],
                                                             out_dtype=BF16),)),
        ("4-bit product", lambda: (tkq.w4_product(d["xq"], d["xs"], d["q32"], d["q32_sf"], d["ids"]),)),
        ("4-bit product, groups of 128", lambda: (tkq.w4_product(d["xq"], d["xs"], d["q128"], d["q128_sf"], d["ids"]),)),
        ("4-bit product of one matrix", lambda: (tkq.w4_product(few, few_sf, d["q32"][0], d["q32_sf"][0]),)),
        ("4-bit cast", lambda: tkq.w4_cast(d["m4"])),
        ("4-bit cast, groups of 128", lambda: tkq.w4_cast(d["m4"], 128)),
    ]


def written(outs):
    return [bits(t).clone() for t in outs if t is not None]


def test_inputs_written_late_on_a_side_stream(cuda_device):
    before, after = inputs(1), inputs(2)
    stale = [written(fn()) for _, fn in calls(before)]
    want = [written(fn()) for _, fn in calls(after)]
    held = {n: t.clone() for n, t in before.items()}
    made = calls(held)
    side, filler = torch.cuda.Stream(), torch.empty(1 << 28, device="cuda")
    for i, (name, fn) in enumerate(made):
        # (rounded up to 128, the experts' starts may agree; the call's other outputs do not)
        assert any(not torch.equal(u, v) for u, v in zip(stale[i], want[i])), f"{name}: the data before gives the same"
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                filler.fill_(float(i))
            for n, t in held.items():
                t.copy_(after[n])
            got = written(fn())
            for n, t in held.items():
                t.copy_(before[n])
        side.synchronize()
        assert len(got) == len(want[i]) and all(torch.equal(u, v) for u, v in zip(got, want[i])), name
    assert tkq.tkq_read_device_status() == 0
