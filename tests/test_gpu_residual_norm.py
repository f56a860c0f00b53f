"""The norms around a block and their gradients against the 64-bit formulas.

Error bounds, u = 2^-24.  A sum over a row adds at most 40 rounded terms in a
row and its squares or products are rounded before: 64 u of the sum of
magnitudes, half of that for the factors p and q.  sigmoid(gate) carries
(2 |gate| + 8) u.  A row's branch a b is within k = (2 |gate| + 60) u of its
magnitude, r' adds u; x adds q's error (its own 40 u, and the row's error
relative to the row).  The gradients are sums of the terms below, taken in
magnitude: 80 u for the stream, 160 u (and the sigmoid's) for the branch, and
one u for each row added to a weight gradient.  bf16 outputs round once (2^-8);
casts as in test_gpu_swiglu_ckpt."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import blocks64 as B
from tests.test_gpu_swiglu_ckpt import _bytes, _check_cast

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


def _inputs(seed, T, C, f32, gated, w_post, w_pre, dev):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)
    r = normal(T, C) * 3
    h = normal(T, C) * 0.7
    h[2::5] = 0                       # a block that gives nothing, a channel far out
    h[::3, 7] *= 40
    r[4::9] = 0
    d = dict(r=r if f32 else r.bfloat16(), h=h.bfloat16(),
             gate=(normal(T, C) * 2).bfloat16() if gated else None,
             w_post=1 + 0.3 * normal(C) if w_post else None,
             w_pre=1 + 0.3 * normal(C) if w_pre else None)
    if gated:
        d["gate"][::4, ::31] = -200.0
        d["gate"][1::4, ::31] = 200.0
    return d, {k: None if v is None else v.to(dev) for k, v in d.items()}


def _64(d):
    return {k: None if v is None else v.double() for k, v in d.items()}


def _forward_reference(d, post, a, eps):
    z = _64(d)
    r, x, p, q = B.residual_norm(z["r"], z["h"], z["w_post"], z["gate"], z["w_pre"], post, a, eps)
    k = 60.0 if z["gate"] is None else 2 * z["gate"].abs() + 60
    b = 0.0 if z["h"] is None else k * U * (r - z["r"]).abs()
    err_r = b + U * r.abs() + TINY
    err_q = 40 * U + err_r.norm(dim=1) / r.norm(dim=1).clamp_min(1e-30)
    wq = 1.0 if z["w_pre"] is None else z["w_pre"].abs()
    err_x = err_r * q[:, None] * wq + (err_q[:, None] + 4 * U) * x.abs()
    return r, err_r, x, err_x, p, q, err_q


CASES = [(1, 128), (4, 7168), (3, 2176), (33, 384), (2, 16384), (70, 1024), (5, 8320)]


@pytest.mark.parametrize("T,C", CASES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("post,gated,w_post,w_pre", [
    (True, True, True, True), (True, False, True, True), (False, True, False, True),
    (False, False, True, False), (True, True, False, False)])
def test_forward(cuda_device, T, C, f32, post, gated, w_post, w_pre):
    host, dev = _inputs(T + C, T, C, f32, gated, w_post, w_pre, cuda_device)
    a, eps = 0.6, 1e-5
    r, err_r, x, err_x, p, q, err_q = _forward_reference(host, post, a, eps)
    for fmt in ("e4m3", "e5m2"):
        got_r, codes, sf, got_x, got_p, got_q = tkq.residual_norm_and_cast(
            **dev, post_norm=post, res_scale=a, eps=eps, fmt=fmt, with_bf16=True)
        assert got_r.dtype == host["r"].dtype
        assert (got_r.cpu().double() - r).abs().le((0 if f32 else BF) * r.abs() + 1.01 * err_r).all()
        assert (got_x.cpu().double() - x).abs().le(BF * x.abs() + 1.01 * err_x).all()
        assert (got_q.cpu().double() - q).abs().le(err_q * q).all()
        if post:
            assert (got_p.cpu().double() - p).abs().le(40 * U * p).all()
        else:
            assert got_p is None
        _check_cast(codes, sf, x, err_x + TINY, fmt)
        # each output alone, and the scale layouts, give the same values
        only = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, eps=eps, fmt=fmt,
                                          use_tma_aligned_col_major_sf=True)
        assert only[3] is None and torch.equal(_bytes(only[1]), _bytes(codes))
        assert torch.equal(only[2][:, :T].t(), sf) and (only[2][:, T:] == 0).all()
        assert torch.equal(_bytes(only[0]), _bytes(got_r)) and torch.equal(only[5], got_q)
    only = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, eps=eps, fmt=None, with_bf16=True)
    assert only[1] is None and only[2] is None and torch.equal(_bytes(only[3]), _bytes(got_x))
    packed = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, eps=eps, fmt="e4m3",
                                        use_packed_ue8m0=True)
    e = packed[2].contiguous().view(torch.uint8).view(T, -1)[:, :C // 128]
    codes, sf = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, eps=eps)[1:3]
    p2 = torch.exp2(e.double() - 127)
    assert (p2 >= sf.double()).all() and (p2 < 2 * sf.double()).all()
    if not w_pre:
        return
    host["w_pre"] = dev["w_pre"] = None
    last = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, eps=eps, fmt=None)
    assert last[1:4] == (None, None, None) and last[5] is None
    assert torch.equal(_bytes(last[0]), _bytes(got_r))


@pytest.mark.parametrize("T,C", CASES)
@pytest.mark.parametrize("f32", [False, True])
def test_norm_before_the_first_block(cuda_device, T, C, f32):
    host, dev = _inputs(T, T, C, f32, False, False, True, cuda_device)
    host["h"] = dev["h"] = None
    r, _, x, err_x, _, q, err_q = _forward_reference(host, False, 1.0, 1e-6)
    got = tkq.residual_norm_and_cast(dev["r"], w_pre=dev["w_pre"], with_bf16=True)
    assert got[0] is dev["r"] and got[4] is None
    assert (got[3].cpu().double() - x).abs().le(BF * x.abs() + 1.01 * err_x).all()
    assert (got[5].cpu().double() - q).abs().le(err_q * q).all()
    _check_cast(got[1], got[2], x, err_x + TINY, "e4m3")


def test_the_cast_is_the_per_token_cast(cuda_device):
    """With an fp32 stream, no block and unit weights x is r q: the codes are those of the
    per-token cast of that fp32 matrix, bit for bit."""
    r = torch.randn(19, 640, device=cuda_device) * 5
    _, codes, sf, _, _, q = tkq.residual_norm_and_cast(r)
    ref, ref_sf = tkq.per_token_cast(r * q[:, None])
    assert torch.equal(_bytes(codes), _bytes(ref)) and torch.equal(sf, ref_sf)


def _backward_reference(d, dr, dx, r1, p, q, a):
    """64-bit gradients and their bounds; p and q are the factors that the kernel is given."""
    z = _64(d)
    g = B.residual_norm_backward(dr, r1, z["h"], dx, z["w_post"], z["gate"], z["w_pre"], p, q, a)
    base = torch.zeros_like(g[0]) if dr is None else dr.abs()
    T = len(base)
    b_pre = None
    if dx is not None:
        n = (r1 * q[:, None]).abs()
        e = dx.abs() * (1.0 if z["w_pre"] is None else z["w_pre"].abs())
        base = base + q[:, None] * (e + n * (e * n).mean(1, keepdim=True))
        b_pre = ((T + 100) * U * dx.abs() * n).sum(0) + TINY
    b_r = 80 * U * base + TINY
    if z["h"] is None:
        return g, (b_r, None, None, None, b_pre)
    m = z["h"].abs() * (1.0 if p is None else p[:, None])
    s = torch.ones_like(m) if z["gate"] is None else torch.sigmoid(z["gate"])
    wide = 160.0 if z["gate"] is None else 160 + 4 * z["gate"].abs()
    wp = 1.0 if z["w_post"] is None else z["w_post"].abs()
    e = abs(a) * base
    b_gate = None if z["gate"] is None else wide * U * e * m * wp * s * (1 - s) + TINY
    b_post = ((T + wide + 100) * U * e * s * m).sum(0) + TINY
    f = wide * U * e * s * wp
    b_h = f if p is None else p[:, None] * (f + m * (f * m).mean(1, keepdim=True))
    return g, (b_r, b_h + TINY, b_gate, b_post, b_pre)


@pytest.mark.parametrize("T,C", CASES + [(400, 256), (1300, 128)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("post,gated,w_post,w_pre,pre,with_dr", [
    (True, True, True, True, True, True), (True, False, True, True, True, True),
    (False, True, True, True, True, False), (False, False, False, False, True, True),
    (True, True, False, False, False, True), (True, False, True, False, False, True)])
def test_backward(cuda_device, T, C, f32, post, gated, w_post, w_pre, pre, with_dr):
    host, dev = _inputs(T * 3 + C, T, C, f32, gated, w_post, w_pre and pre, cuda_device)
    gen = torch.Generator().manual_seed(C)
    dx = (torch.randn(T, C, generator=gen) * 0.5).bfloat16() if pre else None
    dr = torch.randn(T, C, generator=gen).to(host["r"].dtype) if with_dr else None
    a = 0.6
    fwd = tkq.residual_norm_and_cast(**dev, post_norm=post, res_scale=a, fmt=None, with_bf16=pre)
    r1, p, q = fwd[0], fwd[4], fwd[5]

    def up(t):
        return None if t is None else t.to(cuda_device)

    def down(t):
        return None if t is None else t.cpu().double()
    got = tkq.residual_norm_backward(up(dr), r1, dev["h"], up(dx), dev["w_post"], dev["gate"],
                                     dev["w_pre"], p, q, a)
    ref, bound = _backward_reference(host, down(dr), down(dx), down(r1), down(p), down(q), a)
    assert got[0].dtype == host["r"].dtype
    rounds = (0 if f32 else BF, BF, BF, 0, 0)
    for name, t, g, b, rnd in zip(("dr", "dh", "dgate", "dw_post", "dw_pre"), got, ref, bound, rounds):
        if t is None:
            assert {"dgate": not gated, "dw_post": not w_post, "dw_pre": not (w_pre and pre)}[name]
            continue
        err = (t.cpu().double() - g).abs()
        assert err.le(rnd * g.abs() + 1.01 * b).all(), (name, float((err / (rnd * g.abs() + b)).max()))


def test_backward_before_the_first_block(cuda_device):
    host, dev = _inputs(1, 21, 640, True, False, False, True, cuda_device)
    host["h"] = dev["h"] = None
    dx = torch.randn(21, 640).bfloat16()
    q = tkq.residual_norm_and_cast(dev["r"], w_pre=dev["w_pre"])[5]
    for dr in (None, torch.randn(21, 640)):
        got = tkq.residual_norm_backward(None if dr is None else dr.to(cuda_device), dev["r"],
                                         dx=dx.to(cuda_device), w_pre=dev["w_pre"], rstd_pre=q)
        ref, bound = _backward_reference(host, None if dr is None else dr.double(), dx.double(),
                                         host["r"].double(), None, q.cpu().double(), 1.0)
        assert got[1] is None and got[2] is None and got[3] is None
        for t, g, b in ((got[0], ref[0], bound[0]), (got[4], ref[4], bound[4])):
            assert (t.cpu().double() - g).abs().le(b).all()


def test_gradients_against_differences(cuda_device):
    """The kernel's gradients along a direction and the difference quotient of the 64-bit forward.
    The stream is fp32, so r' carries no rounding but the forward's own error, which moves a
    gradient by less than its bound."""
    T, C, a, eps = 6, 512, 0.6, 1e-6
    host, dev = _inputs(3, T, C, True, True, True, True, cuda_device)
    host["h"][2::5] = 0.5                      # no rows of zeros: their factor 1 / sqrt(eps) is steep
    host["r"][4::9] = 1.5
    host["gate"].clamp_(-8, 8)
    dev = {k: v.to(cuda_device) for k, v in host.items()}
    dr, dx = torch.randn(T, C), torch.randn(T, C).bfloat16()
    r1, _, _, _, p, q = tkq.residual_norm_and_cast(**dev, res_scale=a, eps=eps)
    got = tkq.residual_norm_backward(dr.to(cuda_device), r1, dev["h"], dx.to(cuda_device),
                                     dev["w_post"], dev["gate"], dev["w_pre"], p, q, a)
    z = _64(host)
    _, bound = _backward_reference(host, dr.double(), dx.double(), r1.cpu().double(),
                                   p.cpu().double(), q.cpu().double(), a)

    def loss(**kw):
        v = {**z, **kw}
        r, x, _, _ = B.residual_norm(v["r"], v["h"], v["w_post"], v["gate"], v["w_pre"], True, a, eps)
        return (r * dr).sum() + (x * dx).sum()
    gen = torch.Generator().manual_seed(9)
    for i, name in enumerate(("r", "h", "gate", "w_post", "w_pre")):
        v = torch.randn(*z[name].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        slope = (loss(**{name: z[name] + step * v}) - loss(**{name: z[name] - step * v})) / (2 * step)
        g = got[i].cpu().double()
        rnd = BF * g.abs() if got[i].dtype == torch.bfloat16 else 0.0
        tol = ((2 * bound[i] + rnd) * v.abs()).sum() + 1e-6
        assert abs(slope - (g * v).sum()) <= tol, name


def test_repeats_bit_for_bit(cuda_device):
    for T, C in [(1000, 1024), (300, 7168)]:
        _, dev = _inputs(T, T, C, False, True, True, True, cuda_device)
        dx = torch.randn(T, C, device=cuda_device).bfloat16()
        r1, _, _, _, p, q = tkq.residual_norm_and_cast(**dev)
        first = None
        for _ in range(5):
            got = tkq.residual_norm_backward(dx, r1, dev["h"], dx, dev["w_post"], dev["gate"],
                                             dev["w_pre"], p, q)
            first = first or got
            assert all(torch.equal(_bytes(x), _bytes(y)) for x, y in zip(first, got))


def test_workspace_does_not_depend_on_the_grid_override(cuda_device, monkeypatch):
    """The environment variable that sizes grids for another number of SMs changes neither the
    workspace a caller has to bring nor, but for the order of the weight sums, the results."""
    T, C = 700, 1024
    _, dev = _inputs(2, T, C, False, True, True, True, cuda_device)
    dx = torch.randn(T, C, device=cuda_device).bfloat16()
    r1, _, _, _, p, q = tkq.residual_norm_and_cast(**dev)
    args = (dx, r1, dev["h"], dx, dev["w_post"], dev["gate"], dev["w_pre"], p, q)
    ref, size = tkq.residual_norm_backward(*args), tkq.tkq_residual_norm_workspace(T, C)
    for sms in ("3", "1000"):
        monkeypatch.setenv("TKQ_NUM_SMS", sms)
        assert tkq.tkq_residual_norm_workspace(T, C) == size
        got = tkq.residual_norm_backward(*args)
        for a, b in zip(ref[:3], got[:3]):
            assert torch.equal(_bytes(a), _bytes(b))
        for a, b in zip(ref[3:], got[3:]):      # the same terms in another order
            assert (a - b).abs().le(2 * (T + 100) * U * a.abs().max()).all()


@pytest.mark.parametrize("asked,launched", [("3", None), (None, "1000"), ("3", "1000")])
def test_workspace_sized_under_another_override(asked, launched, cuda_device, monkeypatch):
    """A workspace of the size that was asked for is enough when the override changes before the
    launch: more rows than the device has partial rows, and the bytes behind it stay as they were."""
    def override(value):
        if value is None:
            monkeypatch.delenv("TKQ_NUM_SMS", raising=False)
        else:
            monkeypatch.setenv("TKQ_NUM_SMS", value)
    T, C, guard = 5000, 1024, 1 << 16
    dx = torch.randn(T, C, device=cuda_device).bfloat16()
    r = torch.randn(T, C, device=cuda_device).bfloat16()
    q = torch.rand(T, device=cuda_device) + 0.5
    override(None)
    _, _, _, _, ref = tkq.residual_norm_backward(None, r, dx=dx, w_pre=torch.ones(C, device=cuda_device),
                                                 rstd_pre=q)
    override(asked)
    size = tkq.tkq_residual_norm_workspace(T, C)
    assert size < T * 2 * C * 4
    work = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device=cuda_device)
    w, dr, dw = torch.ones(C, device=cuda_device), torch.empty_like(r), torch.empty(C, device=cuda_device)
    override(launched)
    st = tkq.tkq_residual_norm_backward(
        None, dx.data_ptr(), r.data_ptr(), None, None, None, w.data_ptr(), None, q.data_ptr(),
        dr.data_ptr(), None, None, None, dw.data_ptr(), work.data_ptr(), T, C, tkq.NORM_PRE, 1.0,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (work[size:] == 0xA5).all()
    # the same terms in another order: one u for each row, of the sum of magnitudes
    terms = (dx.double() * r.double() * q.double()[:, None]).abs().sum(0)
    assert ((dw - ref).abs().double() <= 2 * (T + 160) * U * terms).all()


def test_offsets_beyond_32_bits(cuda_device):
    T, C, n = 140001, 16384, 21
    _, dev = _inputs(1, n, C, False, True, True, True, cuda_device)
    long = {k: v if v.dim() == 1 else torch.zeros(T, C, dtype=v.dtype, device=cuda_device)
            for k, v in dev.items()}
    for k in ("r", "h", "gate"):
        long[k][-n:] = dev[k]
    big, small = tkq.residual_norm_and_cast(**long), tkq.residual_norm_and_cast(**dev)
    for x, y in zip(big, small):
        if x is not None:
            assert torch.equal(_bytes(x[-n:]), _bytes(y))
    dx = torch.zeros(T, C, dtype=torch.bfloat16, device=cuda_device)
    dx[-n:] = torch.randn(n, C, device=cuda_device)
    grads = [tkq.residual_norm_backward(x, f[0], d["h"], x, d["w_post"], d["gate"], d["w_pre"], f[4], f[5])
             for x, f, d in ((dx, big, long), (dx[-n:].clone(), small, dev))]
    for x, y in zip(grads[0][:3], grads[1][:3]):
        assert torch.equal(_bytes(x[-n:]), _bytes(y))
    for x, y in zip(grads[0][3:], grads[1][3:]):       # the other rows add zeros, in another order
        assert (x - y).abs().le(200 * U * y.abs().max()).all()


def test_no_rows(cuda_device):
    r = torch.empty(0, 256, dtype=torch.bfloat16, device=cuda_device)
    w = torch.ones(256, device=cuda_device)
    out = tkq.residual_norm_and_cast(r, r, w_post=w, w_pre=w)
    assert out[0].shape == (0, 256) and out[1].shape == (0, 256) and out[5].shape == (0,)
    g = tkq.residual_norm_backward(r, r, r, r, w, None, w, out[4], out[5])
    assert g[0].shape == (0, 256) and (g[3] == 0).all() and (g[4] == 0).all()
