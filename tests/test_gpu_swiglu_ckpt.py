"""The SwiGLU with an 8-bit checkpoint, and its backward from it.

Forward: bit for bit the two casts it stands for.  Backward against the 64-bit
formulas on the checkpoint's values.  Error bounds, u = 2^-24: exp(-g) carries
(2 |g| + 4) u (rounded argument, base-2 exponential to 2^-22), the sigmoid 3 u
more, so du = d g s w and y = g s u w are within (2 |g| + 12) u of their
magnitude; dg = d u s (1 + g (1 - s)) w is within (6 |g| + 40) u of
|d u s w| (1 + |g| (1 - s)); dw adds H products, at most H / 32 + 32 of them in
a row.  bf16 outputs round once (2^-8), codes of a cast are within half a step
of value / scale (E4M3: 2^-4 relative, 2^-10 absolute; E5M2: 2^-3, 2^-17), and
a scale carries its group's largest error and 2 u."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import blocks64 as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"e4m3": (2.0 ** -4, 2.0 ** -10, 448.0), "e5m2": (2.0 ** -3, 2.0 ** -17, 57344.0)}


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _x(seed, T, H, dev):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2 * H, generator=gen)
    x[:, :H] *= 2
    x[::5, ::17] *= 30          # outliers, rows of zeros, gates whose exponential overflows
    x[3::7] = 0
    x[1::4, 0] = -120
    return x.bfloat16().to(dev)


SHAPES = [(1, 128), (1, 2048), (2, 1408), (5, 640), (37, 384), (130, 256), (64, 4096), (3, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("fmt,ckpt_fmt", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"),
                                          ("e5m2", "e5m2")])
def test_forward_is_the_two_casts(cuda_device, T, H, weighted, fmt, ckpt_fmt):
    x = _x(T + H, T, H, cuda_device)
    w = torch.rand(T, device=cuda_device) if weighted else None
    for opts in ({}, dict(use_tma_aligned_col_major_sf=True), dict(round_sf=True),
                 dict(use_packed_ue8m0=True, use_tma_aligned_col_major_sf=True)):
        got = tkq.swiglu_forward_cast_and_checkpoint(x, fmt, topk_weights=w, ckpt_fmt=ckpt_fmt, **opts)
        ref = (*tkq.swiglu_forward_and_per_token_cast(x, fmt, topk_weights=w, **opts),
               *tkq.per_token_cast(x, ckpt_fmt))
        for name, a, b in zip(("codes", "scales", "checkpoint", "checkpoint scales"), got, ref):
            assert a.dtype == b.dtype and a.shape == b.shape
            assert torch.equal(_bytes(a), _bytes(b)), f"{name} {opts}"


def _reference(ckpt, sf, dy, w):
    """64-bit dx, dw, y and the bounds of their binary32 evaluation."""
    T, H2 = ckpt.shape
    H = H2 // 2
    x = (ckpt.cpu().float() * sf.cpu().repeat_interleave(128, 1)).double()
    d = dy.cpu().double()
    w64 = None if w is None else w.cpu().double()
    dx, dw = B.swiglu_backward(x, d, w64)
    g, u = x[:, :H], x[:, H:]
    s = torch.sigmoid(g)
    wt = 1.0 if w is None else w64[:, None].abs()
    bound_g = (6 * g.abs() + 40) * U * (d * u).abs() * s * wt * (1 + g.abs() * (1 - s))
    bound_u = (2 * g.abs() + 12) * U * (d * g).abs() * s * wt
    terms = (d * g * s * u).abs()
    bound_w = ((2 * g.abs() + 14 + H / 32 + 32) * U * terms).sum(1)
    y = B.swiglu(x, w64)
    bound_y = (2 * g.abs() + 12) * U * y.abs()
    # below the smallest normal numbers results may be flushed to zero
    return dx, torch.cat([bound_g, bound_u], 1) + 2.0 ** -110, dw, bound_w + 2.0 ** -110, y, bound_y + 2.0 ** -110


def _check_cast(codes, sf, dx, bound, fmt):
    rel, absolute, top = HALF_STEP[fmt]
    groups = dx.abs().view(len(dx), -1, 128)
    s = groups.amax(2).clamp_min(1e-4) / top
    got = sf.cpu().double()
    assert (got - s).abs().le(2 * U * s + bound.view_as(groups).amax(2) / top).all()
    each = got.repeat_interleave(128, 1)
    v = dx / each
    err = (codes.cpu().float().double() - v).abs()
    # the quotient itself: the product by the rounded reciprocal, 2 u, and the value's bound
    slack = bound / each + 4 * U * v.abs()
    assert err.le(torch.maximum(rel * (v.abs() + slack), torch.tensor(absolute)) + slack).all()


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("ckpt_fmt", ["e4m3", "e5m2"])
def test_backward(cuda_device, T, H, weighted, ckpt_fmt):
    dev = cuda_device
    ckpt, sf = tkq.per_token_cast(_x(T * H, T, H, dev), ckpt_fmt)
    gen = torch.Generator().manual_seed(T)
    dy = (torch.randn(T, H, generator=gen) * 0.5).bfloat16().to(dev)
    w = (torch.rand(T, generator=gen) + 0.05).to(dev) if weighted else None
    dx, bx, dw, bw, y, by = _reference(ckpt, sf, dy, w)

    got, none, gw, gy = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, topk_weights=w,
                                                            with_weight_grad=True, with_y=True)
    assert none is None and got.dtype == gy.dtype == torch.bfloat16 and gw.dtype == torch.float32
    assert (got.cpu().double() - dx).abs().le(2.0 ** -8 * dx.abs() + 1.01 * bx).all()
    assert (gy.cpu().double() - y).abs().le(2.0 ** -8 * y.abs() + 1.01 * by).all()
    assert (gw.cpu().double() - dw).abs().le(bw).all()

    for fmt in ("e4m3", "e5m2"):
        codes, s, gw2, gy2 = tkq.swiglu_backward_from_checkpoint(
            ckpt, sf, dy, fmt, topk_weights=w, with_weight_grad=True, with_y=True)
        assert torch.equal(gw2, gw) and torch.equal(_bytes(gy2), _bytes(gy))
        _check_cast(codes, s, dx, bx, fmt)
        # the outputs that are not asked for change nothing
        alone = tkq.swiglu_backward_from_checkpoint(ckpt.view(torch.uint8), sf, dy, fmt,
                                                    topk_weights=w, ckpt_fmt=ckpt_fmt)
        assert alone[2] is None and alone[3] is None
        assert torch.equal(_bytes(alone[0]), _bytes(codes)) and torch.equal(alone[1], s)
        # column-major scales: the same scales and codes, zero padding
        cm = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, fmt, topk_weights=w,
                                                 use_tma_aligned_col_major_sf=True)
        assert torch.equal(_bytes(cm[0]), _bytes(codes)) and torch.equal(cm[1][:, :T].t(), s)
        assert (cm[1][:, T:] == 0).all()
        # powers of two, packed: the scale rounded up, codes of value / that scale
        packed = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, fmt, topk_weights=w,
                                                     use_packed_ue8m0=True)
        e = packed[1].contiguous().view(torch.uint8).view(T, -1)
        G = 2 * H // 128
        p2 = torch.exp2(e[:, :G].double() - 127).cpu()
        assert (e[:, G:] == 0).all()
        assert (p2 >= s.cpu().double()).all() and (p2 < 2 * s.cpu().double()).all()
        rel, absolute, _ = HALF_STEP[fmt]
        v = dx / p2.repeat_interleave(128, 1)
        slack = bx / p2.repeat_interleave(128, 1) + 4 * U * v.abs()
        assert (packed[0].cpu().float().double() - v).abs().le(
            torch.maximum(rel * (v.abs() + slack), torch.tensor(absolute)) + slack).all()


def test_weight_gradient_is_a_difference_quotient(cuda_device):
    """dw along a direction, and the 64-bit forward's difference quotient (linear in w: exact)."""
    T, H = 9, 512
    ckpt, sf = tkq.per_token_cast(_x(2, T, H, cuda_device))
    dy = torch.randn(T, H).bfloat16().to(cuda_device)
    w = torch.rand(T).to(cuda_device)
    dx, _, dw, _ = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, topk_weights=w, with_weight_grad=True)
    ref_dx, bx, _, bw, _, _ = _reference(ckpt, sf, dy, w)
    x = (ckpt.cpu().float() * sf.cpu().repeat_interleave(128, 1)).double()
    d, w64 = dy.cpu().double(), w.cpu().double()
    v = torch.randn(T, dtype=torch.float64)
    slope = ((B.swiglu(x, w64 + v) - B.swiglu(x, w64 - v)) * d).sum() / 2
    assert abs(slope - (dw.cpu().double() * v).sum()) <= (bw * v.abs()).sum() + 1e-9
    # dx: central differences of step h, h^2 times third derivatives of order |x|^3, below 1e-5
    v = torch.randn(T, 2 * H, dtype=torch.float64)
    h = 1e-5
    slope = ((B.swiglu(x + h * v, w64) - B.swiglu(x - h * v, w64)) * d).sum() / (2 * h)
    tol = ((2.0 ** -8 * ref_dx.abs() + 1.01 * bx) * v.abs()).sum() + 1e-5
    assert abs(slope - (dx.cpu().double() * v).sum()) <= tol


def test_repeats_bit_for_bit(cuda_device):
    for T, H in [(3, 7168), (700, 2048), (5000, 1408)]:
        ckpt, sf = tkq.per_token_cast(_x(T, T, H, cuda_device))
        dy = torch.randn(T, H, device=cuda_device).bfloat16()
        a = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, with_weight_grad=True)
        for _ in range(5):
            b = tkq.swiglu_backward_from_checkpoint(ckpt, sf, dy, with_weight_grad=True)
            assert torch.equal(a[2], b[2]) and torch.equal(_bytes(a[0]), _bytes(b[0]))


def test_offsets_beyond_32_bits(cuda_device):
    T, H, n = 140001, 8192, 33       # 2.29e9 elements of x and of dx
    x = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device=cuda_device)
    x[-n:] = _x(1, n, H, cuda_device)
    tail = x[-n:].clone()
    big, small = tkq.swiglu_forward_cast_and_checkpoint(x), tkq.swiglu_forward_cast_and_checkpoint(tail)
    for a, b in zip(big, small):
        assert torch.equal(_bytes(a[-n:]), _bytes(b))
    del x
    dy = torch.randn(n, H, device=cuda_device).bfloat16()
    long = torch.zeros(T, H, dtype=torch.bfloat16, device=cuda_device)
    long[-n:] = dy
    for fmt in (None, "e4m3"):
        a = tkq.swiglu_backward_from_checkpoint(big[2], big[3], long, fmt, with_weight_grad=True, with_y=True)
        b = tkq.swiglu_backward_from_checkpoint(small[2], small[3], dy, fmt, with_weight_grad=True, with_y=True)
        assert torch.equal(_bytes(a[0][-n:]), _bytes(b[0])) and torch.equal(_bytes(a[3][-n:]), _bytes(b[3]))
        if fmt:
            assert torch.equal(a[1][-n:], b[1])
        # the row's sum may be split over more warps in the short call
        _, _, _, bound, _, _ = _reference(small[2], small[3], dy, None)
        assert ((a[2][-n:] - b[2]).abs().cpu().double() <= 2 * bound).all()


def test_no_rows(cuda_device):
    x = torch.empty(0, 512, dtype=torch.bfloat16, device=cuda_device)
    out, sf, ckpt, csf = tkq.swiglu_forward_cast_and_checkpoint(x)
    assert out.shape == (0, 256) and ckpt.shape == (0, 512) and csf.shape == (0, 4)
    dx, _, dw, y = tkq.swiglu_backward_from_checkpoint(ckpt, csf, x[:, :256].contiguous(),
                                                       with_weight_grad=True, with_y=True)
    assert dx.shape == (0, 512) and dw.shape == (0,) and y.shape == (0, 256)
