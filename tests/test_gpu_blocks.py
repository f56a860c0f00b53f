"""The routing, checkpoint and norm calls together: in the access-checked build, captured in a CUDA
graph, on a side stream, and back to back through each other's outputs."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

pytestmark = pytest.mark.gpu

WITHHOLD = 16


@pytest.fixture(scope="module", autouse=True)
def _libraries(cuda_device):
    import __graft_entry__
    from fp8_activation_quantization_gb300 import _build
    __graft_entry__.build()
    _build.build(checked=True)
    tkq.load_library()
    yield


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def _cases(small):
    """(name, fn): fn() makes one call and returns its outputs."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    cases = []
    for T, E, k, groups, dtype in [(1, 256, 8, 8, torch.float32), (37, 60, 4, 1, torch.bfloat16),
                                   (130, 1024, 32, 32, torch.float32), (9, 33, 5, 3, torch.bfloat16)]:
        x = _randn(gen, T, E + 3, dtype=dtype)[:, 2:2 + E]
        bias = _randn(gen, E, dtype=torch.float32) * 0.01
        counts = torch.zeros(E, dtype=torch.int32, device="cuda")
        for scores in ("softmax", "sigmoid"):
            def route(x=x, k=k, groups=groups, bias=bias, counts=counts, scores=scores):
                counts.zero_()
                return (*tkq.route_topk(x, k, scores, bias, groups, max(1, groups // 2), counts=counts),
                        counts)
            cases.append((f"route {T}x{E} {scores}", route))
            ids = tkq.route_topk(x, k, scores)[0]
            dw = _randn(gen, T, k, dtype=torch.float32)
            cases.append((f"route backward {T}x{E} {scores}",
                          lambda x=x, i=ids, d=dw, s=scores: (tkq.route_topk_backward(x, i, d, s),)))
    for T, H, flags in [(1, 128, 0), (7, 1408, 4), (130, 384, 6), (33, 2048, 0)]:
        x = _randn(gen, T, 2 * H)
        w = torch.rand(T, generator=gen, device="cuda")
        opts = dict(use_packed_ue8m0=bool(flags & 2), use_tma_aligned_col_major_sf=bool(flags & 4))
        cases.append((f"save {T}x{H} {flags}", lambda x=x, w=w, o=opts:
                      tkq.swiglu_forward_cast_and_checkpoint(x, "e4m3", topk_weights=w, ckpt_fmt="e5m2", **o)))
        ck, sf = tkq.per_token_cast(x)
        dy = _randn(gen, T, H)
        for fmt in (None, "e4m3"):
            cases.append((f"restore {T}x{H} {fmt} {flags}", lambda c=ck, s=sf, d=dy, f=fmt, w=w, o=opts:
                          tuple(t for t in tkq.swiglu_backward_from_checkpoint(
                              c, s, d, f, topk_weights=w, with_weight_grad=True, with_y=True,
                              **(o if f else {})) if t is not None)))
    for T, C, f32, flags in [(1, 128, False, 0), (5, 7168, False, 4), (33, 640, True, 6), (2, 16384, True, 0)]:
        res = torch.float32 if f32 else torch.bfloat16
        r, h, gate = _randn(gen, T, C, dtype=res), _randn(gen, T, C), _randn(gen, T, C)
        wp, wq = torch.rand(C, generator=gen, device="cuda"), torch.rand(C, generator=gen, device="cuda")
        opts = dict(use_packed_ue8m0=bool(flags & 2), use_tma_aligned_col_major_sf=bool(flags & 4))
        cases.append((f"norm {T}x{C} {flags}", lambda r=r, h=h, g=gate, p=wp, q=wq, o=opts:
                      tkq.residual_norm_and_cast(r, h, p, g, q, with_bf16=True, **o)))
        _, _, _, _, p, q = tkq.residual_norm_and_cast(r, h, wp, gate, wq)
        dx, dr = _randn(gen, T, C), _randn(gen, T, C, dtype=res)
        cases.append((f"norm backward {T}x{C}",
                      lambda r=r, h=h, g=gate, wp=wp, wq=wq, p=p, q=q, dx=dx, dr=dr:
                      tkq.residual_norm_backward(dr, r, h, dx, wp, g, wq, p, q, 0.5)))
    return cases[::3] if small else cases


def test_every_call_stays_inside_its_buffers(cuda_device):
    for name, fn in _cases(False):
        ref = [_bytes(t) for t in fn()]
        with tkq.use_checked_library():
            tkq.tkq_read_device_status(clear=True)
            tkq.tkq_read_check_address(clear=True)
            got = [_bytes(t) for t in fn()]
            status = tkq.tkq_read_device_status(clear=True)
            bad = tkq.tkq_read_check_address(clear=True)
        assert status == 0 and bad == 0, f"{name}: status {status}, refused address {bad:#x}"
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a, b), f"{name}: output {i} differs from the release build"


def test_withheld_output_tails_are_refused_and_reported(cuda_device, monkeypatch):
    cases = _cases(False)
    monkeypatch.setenv("TKQ_CHECK_WITHHOLD", str(WITHHOLD))
    with tkq.use_checked_library():
        for name, fn in cases:
            tkq.tkq_read_device_status(clear=True)
            tkq.tkq_read_check_address(clear=True)
            fn()
            status = tkq.tkq_read_device_status(clear=True)
            bad = tkq.tkq_read_check_address(clear=True)
            assert status & tkq.DEVICE_OUT_OF_BOUNDS, f"{name}: no refused access reported"
            assert bad, f"{name}: no address"


def test_graph_replay_and_side_streams_match_direct_calls(cuda_device):
    cases = _cases(False)
    ref = [[_bytes(t).clone() for t in fn()] for _, fn in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = [[_bytes(t).clone() for t in fn()] for _, fn in cases]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [[t for t in fn()] for _, fn in cases]
    for _ in range(3):
        for t in (t for o in outs for t in o):
            _bytes(t).zero_()
        g.replay()
        torch.cuda.synchronize()
        for (name, _), a, b, c in zip(cases, ref, outs, other):
            for i, (x, y, z) in enumerate(zip(a, b, c)):
                if name.startswith("route ") and i == 2:
                    continue                       # one counter for direct calls and replays
                assert torch.equal(x, _bytes(y)), f"{name}: output {i} of the replay"
                assert torch.equal(x, z), f"{name}: output {i} on another stream"
    assert tkq.tkq_read_device_status() == 0


def test_chained_calls_see_each_others_results(cuda_device):
    """norm -> cast back -> save -> restore -> norm backward, again and again without a wait, the
    buffers of one round reused by the next."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, H = 257, 1024
    rs = [_randn(gen, T, 2 * H) for _ in range(4)]
    h, dy, w = _randn(gen, T, 2 * H), _randn(gen, T, H), torch.rand(2 * H, generator=gen, device="cuda")

    def chain(r, wait):
        def step(v):
            if wait:
                torch.cuda.synchronize()
            return v
        r1, q, sf, _, p, s = step(tkq.residual_norm_and_cast(r, h, w, None, w))
        x = step(tkq.cast_back(q, sf, out_dtype=torch.bfloat16))
        _, _, ck, csf = step(tkq.swiglu_forward_cast_and_checkpoint(x))
        dx, _, dw, _ = step(tkq.swiglu_backward_from_checkpoint(ck, csf, dy, with_weight_grad=True))
        ids, _ = step(tkq.route_topk(x[:, :100], 6))
        dl = step(tkq.route_topk_backward(x[:, :100], ids, dw[:, None].expand(-1, 6).contiguous()))
        return [*step(tkq.residual_norm_backward(r, r1, h, dx, w, None, w, p, s)), dw, dl]

    ref = [[None if t is None else _bytes(t).clone() for t in chain(r, True)] for r in rs]
    for _ in range(10):
        for r, want in zip(rs, ref):
            for a, b in zip(chain(r, False), want):
                assert a is None or torch.equal(_bytes(a), b)
