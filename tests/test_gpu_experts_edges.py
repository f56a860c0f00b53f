"""The experts' operators where calls meet their surroundings: the access-checked build, graphs, streams, two
calls at once, grids that pass over their work many times, more than 2^31 elements, and a whole training step
of them together."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
WITHHOLD = 16

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    from fp8_activation_quantization_gb300 import _build
    __graft_entry__.build()
    _build.build(checked=True)


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def ids_of(T, k, E, g, empty=0.1):
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    return torch.where(torch.rand(T, k, generator=g, device="cuda") < empty, -1, ids).contiguous()


def codes(rows, cols, g):
    return tkq.per_token_cast(torch.randn(rows, cols, generator=g, device="cuda").bfloat16())


def bits(t):
    return t.contiguous().view(torch.uint8)


def cases(T=70, C=384, E=7, k=3, align=128, N=256, seed=0):
    """(name, call) of every entry point; a call returns the tensors it wrote.  Rows that a call leaves as they
    were are in buffers of zeros."""
    g = gen(seed)
    dev = "cuda"
    ids = ids_of(T, k, E, g)
    order = tkq.expert_order(ids, E, align)
    R = order.rows.numel()
    x = torch.randn(T, C, generator=g, device=dev).bfloat16()
    xq, xs = tkq.per_token_cast(x, "e5m2")
    w = torch.rand(T, k, generator=g, device=dev)
    y = torch.randn(R, C, generator=g, device=dev).bfloat16()
    a, a_sf = codes(R, C, g)
    m = [tkq.per_block_cast(torch.randn(N, C, generator=g, device=dev).bfloat16()) for _ in range(E)]
    mw, ms = torch.stack([bits(v[0]) for v in m]).view(F8), torch.stack([v[1] for v in m])
    R128 = -(-R // 128) * 128
    starts = torch.arange(E + 1, dtype=torch.int32, device=dev) * (R128 // 128 // E) * 128
    t1 = tkq.per_channel_cast(torch.randn(R128, N, generator=g, device=dev).bfloat16(), transpose=True)
    t2 = tkq.per_channel_cast(torch.randn(R128, C, generator=g, device=dev).bfloat16(), transpose=True)
    q, qs = tkq.w4_cast(torch.randn(E, N, C, generator=g, device=dev).bfloat16())
    q2, q2s = tkq.w4_cast(torch.randn(N, C, generator=g, device=dev).bfloat16(), 128)
    xe, xes = codes(T * k, C, g)
    x4, x4s = tkq.per_token_cast(x)
    zero = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device=dev)
    rows = lambda r: tkq.ExpertOrder(r[0], r[1], r[2])
    return [
        ("order", lambda: tuple(tkq.expert_order(ids, E, align))),
        ("gather bf16", lambda: [v for v in tkq.expert_gather(x, order, weights=w, out=zero(R, C, dtype=BF16),
                                                              row_weights=zero(R, dtype=F32)) if v is not None]),
        ("gather cast", lambda: tkq.expert_gather(x, order, "e4m3", weights=w, out=zero(R, C), out_sf=zero(R, C // 128, dtype=F32),
                                                  row_weights=zero(R, dtype=F32))),
        ("gather codes", lambda: tkq.expert_gather(xq, order, x_sf=xs, out=zero(R, C), out_sf=zero(R, C // 128, dtype=F32))[:2]),
        ("reduce", lambda: tkq.expert_reduce(y, rows(order), w, y[:, 0].float().contiguous())),
        ("reduce fp32", lambda: tkq.expert_reduce(y, order, out_dtype=F32)[:1]),
        ("reduce backward", lambda: [v for v in tkq.expert_reduce_backward(x, y, order, w, out=zero(R, C, dtype=BF16)) if v is not None]),
        ("reduce backward cast", lambda: tkq.expert_reduce_backward(x, y, order, w, "e4m3", out=zero(R, C),
                                                                    out_sf=zero(R, C // 128, dtype=F32))),
        ("product", lambda: (tkq.expert_product(a, a_sf, mw, ms, order.offsets, out=zero(R, N, dtype=BF16)),)),
        ("weight grad", lambda: (tkq.expert_weight_grad(*t1, *t2, starts),)),
        ("weight grad bf16", lambda: (tkq.expert_weight_grad(*t1, *t2, starts, out_dtype=BF16),)),
        ("w4 experts", lambda: (tkq.w4_product(xe, xes, q, qs, ids),)),
        ("w4 shared rows", lambda: (tkq.w4_product(x4, x4s, q, qs, ids),)),
        ("w4 one matrix", lambda: (tkq.w4_product(xe[:5], xes[:5], q2, q2s),)),
        ("w4 cast", lambda: tkq.w4_cast(x, 32)),
        ("w4 cast 128", lambda: tkq.w4_cast(x, 128)),
    ]


def last_store_is_withheld(name):
    """Whether the call writes its outputs' last bytes (rows from the last expert's end on are not written)."""
    return name in ("order", "reduce", "reduce fp32", "weight grad", "weight grad bf16", "w4 experts", "w4 shared rows",
                    "w4 one matrix", "w4 cast", "w4 cast 128")


@pytest.mark.parametrize("shape", [dict(), dict(T=1, C=128, E=3, k=2, align=1, N=128), dict(T=131, C=1408, E=5, k=4, align=16, N=384)])
def test_every_entry_point_stays_inside_its_buffers(cuda_device, shape):
    for name, fn in cases(**shape):
        ref = [bits(t).clone() for t in fn()]
        with tkq.use_checked_library():
            tkq.tkq_read_device_status(clear=True)
            tkq.tkq_read_check_address(clear=True)
            got = [bits(t).clone() for t in fn()]
            status, bad = tkq.tkq_read_device_status(clear=True), tkq.tkq_read_check_address(clear=True)
        assert status == 0 and bad == 0, f"{name}: status {status}, refused address {bad:#x}"
        for i, (u, v) in enumerate(zip(got, ref)):
            assert torch.equal(u, v), f"{name}: output {i} differs from the release build"


def test_withheld_output_tails_are_refused_and_reported(cuda_device, monkeypatch):
    made = cases()
    monkeypatch.setenv("TKQ_CHECK_WITHHOLD", str(WITHHOLD))
    with tkq.use_checked_library():
        tkq.tkq_read_device_status(clear=True)
        tkq.tkq_read_check_address(clear=True)
        for name, fn in made:
            outs = fn()
            status, bad = tkq.tkq_read_device_status(clear=True), tkq.tkq_read_check_address(clear=True)
            if not last_store_is_withheld(name):
                continue
            assert status & tkq.DEVICE_OUT_OF_BOUNDS, f"{name}: no refused access reported"
            assert bad >> 63 == 1, f"{name}: the refused access is not a store ({bad:#x})"
            addr = bad & ((1 << 63) - 1)
            ends = [t.data_ptr() + t.numel() * t.element_size() for t in outs if t is not None]
            assert any(e - WITHHOLD <= addr < e for e in ends), f"{name}: {addr:#x}"


@pytest.mark.parametrize("sms", [1, 3])
def test_small_grids_give_the_same_bytes(cuda_device, monkeypatch, sms):
    for name, fn in cases(T=250, C=640, E=9, k=4, align=16, N=640):
        ref = [bits(t).clone() for t in fn()]
        monkeypatch.setenv("TKQ_NUM_SMS", str(sms))
        got = [bits(t).clone() for t in fn()]
        monkeypatch.delenv("TKQ_NUM_SMS")
        for i, (u, v) in enumerate(zip(got, ref)):
            assert torch.equal(u, v), f"{name}: output {i}"


def test_captured_and_replayed(cuda_device):
    """A graph of the whole chain, replayed on other inputs in the same tensors, twice each."""
    T, k, E, C, N = 90, 4, 12, 384, 256
    g = gen(3)
    fresh = lambda s: (ids_of(T, k, E, gen(s)), torch.randn(T, C, generator=gen(s + 1), device="cuda").bfloat16(),
                       torch.rand(T, k, generator=gen(s + 2), device="cuda"))
    m = [tkq.per_block_cast(torch.randn(N, C, generator=g, device="cuda").bfloat16()) for _ in range(E)]
    mw, ms = torch.stack([bits(v[0]) for v in m]).view(F8), torch.stack([v[1] for v in m])
    q, qs = tkq.w4_cast(torch.randn(E, N, C, generator=g, device="cuda").bfloat16())
    held = [t.clone() for t in fresh(10)]

    def chain(ids, x, w):
        order = tkq.expert_order(ids, E)
        a, a_sf, rw = tkq.expert_gather(x, order, "e4m3", weights=w)
        y = tkq.expert_product(a, a_sf, mw, ms, order.offsets)
        out, values = tkq.expert_reduce(y, order, w, rw)
        dy, _, dw = tkq.expert_reduce_backward(out, y, order, w, out=torch.zeros_like(y))
        grad = tkq.expert_weight_grad(*tkq.per_channel_cast(dy, transpose=True),
                                      *tkq.per_channel_cast(torch.zeros_like(dy), transpose=True), order.offsets)
        few = tkq.w4_product(*tkq.per_token_cast(x), q, qs, ids)
        return order.slots, out, values, dw, grad, few

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(*held)
    for s in (20, 30, 20):
        for to, new in zip(held, fresh(s)):
            to.copy_(new)
        want = [t.clone() for t in chain(*held)]
        for _ in range(2):
            graph.replay()
            for i, (u, v) in enumerate(zip(outs, want)):
                assert torch.equal(bits(u), bits(v)), i
    assert tkq.tkq_read_device_status() == 0


def test_an_order_of_a_whole_cluster_captured_and_replayed(cuda_device):
    T, k, E = 5000, 8, 100
    ids = ids_of(T, k, E, gen(1))
    order = tkq.expert_order(ids, E)                 # its buffers are the graph's
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tkq.expert_order(ids, E, 128, *order)
    for s in (2, 3):
        ids.copy_(ids_of(T, k, E, gen(s)))
        graph.replay()
        for u, v in zip(order, tkq.expert_order(ids, E)):
            assert torch.equal(u, v)


def test_on_a_side_stream_behind_its_work(cuda_device):
    """Calls go to the current stream: inputs are written there just before, late."""
    side = torch.cuda.Stream()
    late = torch.empty(1 << 28, device="cuda")
    made = cases(seed=4)
    want = [[bits(t).clone() for t in fn()] for _, fn in made]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = []
        for _, fn in made:
            late.fill_(1.0)
            got.append([bits(t) for t in fn()])
    side.synchronize()
    for (name, _), a, b in zip(made, got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b)), name


def test_two_calls_at_once(cuda_device):
    """The same entry points on two streams at the same time, on different tensors."""
    one, two = cases(T=256, C=1024, E=16, k=4, N=1024, seed=5), cases(T=500, C=640, E=5, k=2, N=896, seed=6)
    want = [[bits(t).clone() for t in fn()] for _, fn in one + two]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[] for _ in one + two]
    for _ in range(5):
        for i in range(len(one)):
            for s, (st, made) in enumerate(zip(streams, (one, two))):
                with torch.cuda.stream(st):
                    got[s * len(one) + i] = made[i][1]()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert all(torch.equal(bits(u), v) for u, v in zip(a, b)), (one + two)[i][0]
    assert tkq.tkq_read_device_status() == 0


def test_empty_batches(cuda_device):
    dev = "cuda"
    order = tkq.expert_order(torch.empty(0, 4, dtype=torch.int32, device=dev), 6)
    assert order.rows.numel() == 0 and not bool(order.offsets.any())
    x = torch.empty(0, 256, dtype=BF16, device=dev)
    w = torch.empty(0, 4, device=dev)
    assert tkq.expert_gather(x, order, "e4m3", weights=w)[0].shape == (0, 256)
    assert tkq.expert_reduce(x, order, w, torch.empty(0, device=dev))[1].shape == (0, 4)
    assert tkq.expert_reduce_backward(x, x, order, w)[2].shape == (0, 4)
    f8 = lambda *s: torch.empty(*s, dtype=F8, device=dev)
    assert tkq.expert_product(f8(0, 256), torch.empty(0, 2, device=dev), f8(6, 128, 256), torch.ones(6, 1, 2, device=dev),
                              order.offsets).shape == (0, 128)
    assert tkq.w4_product(f8(0, 256), torch.empty(0, 2, device=dev), torch.zeros(128, 128, dtype=torch.uint8, device=dev),
                          torch.zeros(128, 8, dtype=torch.uint8, device=dev)).shape == (0, 128)
    # tokens of which none has an expert: no rows, sums of nothing
    order = tkq.expert_order(torch.full((9, 4), -1, dtype=torch.int32, device=dev), 6, 16)
    x = torch.randn(9, 256, device=dev).bfloat16()
    y, _, rw = tkq.expert_gather(x, order, weights=torch.rand(9, 4, device=dev))
    out, values = tkq.expert_reduce(y, order, torch.rand(9, 4, device=dev), rw)
    assert not bool(out.any()) and not bool(values.any())
    assert not bool(tkq.expert_reduce_backward(x, y, order, torch.rand(9, 4, device=dev))[2].any())


def test_more_than_2_31_elements_of_rows(cuda_device):
    """Rows beyond 2^31 elements: a few tokens at the first and last places."""
    C, T, k = 16384, 20000, 8                        # 2.6e9 codes
    g = gen(7)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[:] = torch.arange(k, device="cuda", dtype=torch.int32)
    order = tkq.expert_order(ids, k, 1)
    x = torch.randn(T, C, generator=g, device="cuda").bfloat16()
    out, sf, _ = tkq.expert_gather(x, order, "e4m3")
    ref, ref_sf = tkq.per_token_cast(x)
    for e in (0, 6, 7):
        for t in (0, 1, T - 1):
            r = e * T + t
            assert torch.equal(bits(out[r]), bits(ref[t])) and torch.equal(sf[r], ref_sf[t])
    del out, sf
    y, _, _ = tkq.expert_gather(x, order)
    back, _ = tkq.expert_reduce(y, order, out_dtype=F32)
    for t in (0, 77, T - 1):
        assert torch.equal(back[t], 8 * x[t].float())
    w = torch.full((T, k), 0.5, device="cuda")
    dy, _, dw = tkq.expert_reduce_backward(x, y, order, w, out=y.clone())
    assert torch.equal(dy[7 * T + T - 1].float(), 0.5 * x[T - 1].float())
    ref = x[T - 1].double().square().sum()
    assert abs(float(dw[T - 1, 7] - ref)) <= (8 * 16 + 10) * 2.0 ** -24 * float(ref)


def test_more_than_2_31_elements_in_products(cuda_device):
    R, K, N = 2200000, 1024, 128                     # 2.25e9 codes of a
    one = torch.full((1, K), 0x38, dtype=torch.uint8, device="cuda").view(F8)  # 1.0
    a = one.view(torch.uint8).expand(R, K).contiguous().view(F8)
    a_sf = torch.ones(R, K // 128, device="cuda")
    a_sf[-1] = 2.0
    w = one.view(torch.uint8).expand(2, N, K).contiguous().view(F8)
    w_sf = torch.tensor([1.0, 0.5], device="cuda").view(2, 1, 1).expand(2, 1, K // 128).contiguous()
    out = tkq.expert_product(a, a_sf, w, w_sf, torch.tensor([0, R - 130, R], dtype=torch.int32, device="cuda"))
    for r, v in ((0, 1024.0), (R // 2, 1024.0), (R - 131, 1024.0), (R - 130, 512.0), (R - 2, 512.0), (R - 1, 1024.0)):
        assert bool((out[r] == v).all()), r
    del a, a_sf, out
    R = 17 * 2 ** 20                                 # 2.28e9 codes of each operand
    t = one.view(torch.uint8)[0, :1].expand(128, R).contiguous().view(F8)
    sf = torch.ones(128, R // 128, device="cuda")
    sf[:, -1] = 3.0
    dw = tkq.expert_weight_grad(t, sf, t, sf, torch.tensor([0, R - 256, R], dtype=torch.int32, device="cuda"))
    assert bool((dw[1] == 128 + 9 * 128).all()) and bool((dw[0] == float(R - 256)).all())


def test_more_than_2_31_bytes_of_4_bit_weights(cuda_device):
    E, N, K = 130, 4096, 8192                        # 2.18e9 bytes
    w = torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")      # 1.0
    w[-1] = 0x44                                                                # 2.0
    ws = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    x = torch.full((2, K), 0x38, dtype=torch.uint8, device="cuda").view(F8)
    ids = torch.tensor([[0, E - 1], [E - 1, 64]], dtype=torch.int32, device="cuda")
    out = tkq.w4_product(x, torch.ones(2, K // 128, device="cuda"), w, ws, ids)
    assert [float(v) for v in out[:, -1]] == [8192.0, 16384.0, 16384.0, 8192.0]
    assert bool((out == out[:, :1]).all())


@pytest.mark.parametrize("tokens,channels,hidden,experts,k", [(512, 512, 256, 8, 2), (301, 640, 384, 12, 4), (64, 256, 128, 40, 3)])
def test_training_step_with_fp8_products(cuda_device, tokens, channels, hidden, experts, k):
    """The example's step with every product in FP8, against autograd in binary32.  A cast to E4M3 is off by at
    most 2^-4 of a value, 2^-4 / sqrt(3) = 3.6 % in the root mean square, each independent of the others.  The
    stream passes four (input, w1, activations, w2); a gradient at most eight more (its own rows, w2, its row
    after the SwiGLU and w1; and the checkpoint's gate and up, each made of the first two): 3.6 % sqrt(12) =
    12.5 %, and bf16 roundings.  Bound: 14 %."""
    import moe_block
    errors, saved = moe_block.step(tokens, channels, hidden, experts, k, fp8=True)
    assert int(saved["order"].offsets[-1]) >= tokens * k
    errors.pop("d router")
    for name, e in errors.items():
        assert e < 0.14, f"{name}: {e:.3f}"
    assert tkq.tkq_read_device_status() == 0
