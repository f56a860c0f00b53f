"""Stores at the very end of every output of the experts' operators in the access-checked build: with the last
bytes of the outputs withheld from the table of the call's buffers, each call reports a refused store there, and
every other byte is that of the release build.  Whole orders (one row a pair, none that pads), so every call
writes its outputs' last bytes; the rows' product by boxes of 32 whole rows and by rows of a partial tile."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
WITHHOLD = 4


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    from fp8_activation_quantization_gb300 import _build
    __graft_entry__.build()
    _build.build(checked=True)


def made(T, k, E, C, N):
    """(name, call) of the calls that leave rows behind the last expert's as they were."""
    g = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    order = tkq.expert_order(ids, E, 1)
    R = T * k
    assert int(order.offsets[-1]) == R == order.rows.numel()
    x, y, w = normal(T, C).bfloat16(), normal(R, C).bfloat16(), torch.rand(T, k, generator=g, device="cuda")
    xq, xs = tkq.per_token_cast(x)
    a, a_sf = tkq.per_token_cast(normal(R, C).bfloat16())
    parts = [tkq.per_block_cast(normal(N, C).bfloat16()) for _ in range(E)]
    mw, ms = torch.stack([p[0].view(torch.uint8) for p in parts]).view(F8), torch.stack([p[1] for p in parts])
    zero = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")
    sf = lambda: zero(R, C // 128, dtype=torch.float32)
    rw = lambda: zero(R, dtype=torch.float32)
    return [
        ("gather bf16", lambda: tkq.expert_gather(x, order, out=zero(R, C, dtype=BF16))),
        ("gather bf16, weights", lambda: tkq.expert_gather(x, order, weights=w, out=zero(R, C, dtype=BF16), row_weights=rw())),
        ("gather cast", lambda: tkq.expert_gather(x, order, "e5m2", out=zero(R, C), out_sf=sf())),
        ("gather codes", lambda: tkq.expert_gather(xq, order, x_sf=xs, out=zero(R, C), out_sf=sf())),
        ("reduce backward", lambda: tkq.expert_reduce_backward(x, y, order, w, out=zero(R, C, dtype=BF16))),
        ("reduce backward cast", lambda: tkq.expert_reduce_backward(x, y, order, w, "e4m3", out=zero(R, C), out_sf=sf())),
        ("product", lambda: (tkq.expert_product(a, a_sf, mw, ms, order.offsets, out=zero(R, N, dtype=BF16)),)),
    ]


@pytest.mark.parametrize("T,k,E,C,N", [(64, 1, 1, 256, 256), (256, 1, 1, 128, 384), (50, 3, 5, 384, 128), (129, 2, 2, 256, 256)])
def test_the_last_bytes_of_every_output(cuda_device, monkeypatch, T, k, E, C, N):
    for name, fn in made(T, k, E, C, N):
        want = [t.contiguous().view(torch.uint8).flatten().clone() for t in fn() if t is not None]
        with tkq.use_checked_library():
            tkq.tkq_read_device_status(clear=True)
            tkq.tkq_read_check_address(clear=True)
            outs = [t for t in fn() if t is not None]
            status, bad = tkq.tkq_read_device_status(clear=True), tkq.tkq_read_check_address(clear=True)
            assert status == 0 and bad == 0, f"{name}: {status} {bad:#x}"
            assert all(torch.equal(t.view(torch.uint8).flatten(), v) for t, v in zip(outs, want)), name
            monkeypatch.setenv("TKQ_CHECK_WITHHOLD", str(WITHHOLD))
            outs = [t for t in fn() if t is not None]
            status, bad = tkq.tkq_read_device_status(clear=True), tkq.tkq_read_check_address(clear=True)
            monkeypatch.delenv("TKQ_CHECK_WITHHOLD")
        assert status & tkq.DEVICE_OUT_OF_BOUNDS, f"{name}: no refused access reported"
        assert bad >> 63 == 1, f"{name}: the refused access is not a store ({bad:#x})"
        addr = bad & ((1 << 63) - 1)
        ends = [t.data_ptr() + t.numel() * t.element_size() for t in outs]
        assert any(e - WITHHOLD <= addr < e for e in ends), f"{name}: {addr:#x}"
        for i, (t, v) in enumerate(zip(outs, want)):
            got = t.view(torch.uint8).flatten()
            # a refused store is left out as a whole, 32 bytes at the most
            assert torch.equal(got[:-32], v[:-32]), f"{name}: output {i}"
            if not (name.startswith("reduce backward") and t is outs[-1]):  # dweights is no buffer of zeros
                assert not bool(got[-WITHHOLD:].any()), f"{name}: output {i}: stored where it was withheld"
