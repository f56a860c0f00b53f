"""Expert routing and its gradient against the 64-bit formulas.

Error bounds, u = 2^-24: a score is a sum of at most 37 rounded additions of
exponentials (2 ulp each) whose arguments carry |x - m| u, one division, the
renormalisation a five-level sum and a division, the scale one product; with
`spread` the largest |x - m| (0 for the sigmoid, whose argument is exact) the
relative error of a weight is below (2 spread + 64) u.  A gradient adds two
such sums and products of the terms it is made of: (2 spread + 96) u of the sum
of their magnitudes; bf16 gradients round once, 2^-8 relative.
Choices are compared as whole numbers on rows in which no two keys (or group
scores) are nearer than 2^-18 relative without being equal."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import blocks64 as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


def _decided(x, case, bias):
    """Rows whose order does not hang on the last bits of a score."""
    _, key = B.keys(x.double(), case["kind"], None if bias is None else bias.double())
    lists = [key]
    G = case.get("groups", 1)
    if G > 1:
        two = key.view(len(x), G, -1).sort(2, descending=True).values[:, :, :case.get("group_top", 2)]
        lists.append(two.nan_to_num(neginf=0.0).sum(2))
    ok = torch.ones(len(x), dtype=torch.bool)
    for v in lists:
        v = v.sort(1, descending=True).values
        gap = (v[:, :-1] - v[:, 1:]).nan_to_num(0.0)
        near = (gap > 0) & (gap < 2.0 ** -18 * v[:, :-1].abs()) & torch.isfinite(v[:, :-1])
        ok &= ~near.any(1)
    return ok


def _logits(seed, T, case, dtype, mask=None, bias=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, case["E"], generator=gen) * 2
    for _ in range(50):
        x = x.to(dtype).float()
        if mask is not None:
            mask(x)
        ok = _decided(x, case, bias)
        if ok.all():
            return x.to(dtype)
        x[~ok] = (torch.randn(T, case["E"], generator=gen) * 2)[~ok]
    raise AssertionError("no decided rows drawn")


def _spread(x, kind):
    if kind == "sigmoid":
        return 0.0
    x = torch.where(x > -INF, x.double().clamp(max=B.LARGEST), NAN)
    return float(min(104.0, (x.nan_to_num(-INF).amax(1) - x.nan_to_num(INF).amin(1)).clamp(min=0).max()))


def _check_forward(x, dev, kind, k, bias=None, logits=None, **kw):
    ref_ids, ref_w = B.route(x.double(), k, kind, None if bias is None else bias.double(), **kw)
    counts = torch.zeros(x.shape[1], dtype=torch.int32, device=dev)
    ids, w = tkq.route_topk(x.to(dev) if logits is None else logits, k, scores=kind,
                            bias=None if bias is None else bias.to(dev),
                            num_groups=kw.get("groups", 1), topk_groups=kw.get("topk_groups", 1),
                            num_topk_sum=kw.get("group_top", 2),
                            renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0),
                            counts=counts)
    assert torch.equal(ids.cpu(), ref_ids)
    got = w.cpu().double()
    tol = (2 * _spread(x, kind) + 64) * U
    assert (got - ref_w).abs().le(tol * ref_w.abs() + 2.0 ** -126 * abs(kw.get("scale", 1.0))).all()
    taken = ref_ids[ref_ids >= 0].long()
    assert torch.equal(counts.cpu().long(), torch.bincount(taken, minlength=x.shape[1]))
    return ids, w


@pytest.mark.parametrize("T", [1, 3, 37])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (32, 4), (33, 8), (60, 4), (64, 32),
                                 (160, 6), (256, 8), (257, 9), (1000, 11), (1024, 32)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_sizes(cuda_device, T, E, k, kind):
    for dtype in (torch.bfloat16, torch.float32):
        x = _logits(E + T, T, dict(E=E, kind=kind), dtype)
        for renorm in (False, True):
            _check_forward(x, cuda_device, kind, k, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,topk_groups,group_top,k", [
    (256, 8, 4, 2, 8), (256, 8, 1, 2, 8), (64, 8, 3, 1, 6), (24, 4, 2, 2, 5), (32, 32, 5, 2, 8),
    (160, 8, 3, 2, 6), (60, 4, 4, 2, 7), (36, 3, 2, 1, 30), (1024, 32, 6, 2, 32), (9, 3, 1, 2, 5)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_groups_and_bias(cuda_device, E, groups, topk_groups, group_top, k, kind):
    """Among them k larger than the kept groups hold: the rest is -1."""
    gen = torch.Generator().manual_seed(E)
    for biased in (False, True):
        bias = torch.randn(E, generator=gen) * (0.05 if kind == "sigmoid" else 0.5 / E) if biased else None
        case = dict(E=E, kind=kind, groups=groups, group_top=group_top)
        x = _logits(E + k, 29, case, torch.float32, bias=bias)
        _check_forward(x, cuda_device, kind, k, bias, groups=groups, topk_groups=topk_groups,
                       group_top=group_top, renorm=True)


def _holes(x):
    """Absent experts: some of every row, whole rows, NaN, all but one; the type's lowest value and
    +inf, which are logits."""
    x[:, 1::5] = -INF
    x[2::7] = -INF
    x[3::7] = NAN
    x[4::7, 1:] = -INF
    x[5::7, ::2] = NAN
    x[6::7, 0] = torch.finfo(torch.bfloat16).min
    x[6::7, 2] = INF


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,k", [(40, 1, 6), (40, 4, 6), (256, 8, 16)])
def test_absent_experts(cuda_device, kind, E, groups, k):
    for dtype in (torch.bfloat16, torch.float32):
        case = dict(E=E, kind=kind, groups=groups)
        x = _logits(5, 43, case, dtype, mask=_holes)
        for renorm in (False, True):
            _, w = _check_forward(x, cuda_device, kind, k, groups=groups,
                                  topk_groups=max(1, groups // 2), renorm=renorm)
            assert torch.isfinite(w).all()
    bias = torch.zeros(E)
    bias[3], bias[7], bias[0] = -INF, NAN, INF
    x = _logits(6, 11, dict(E=E, kind=kind), torch.float32, bias=bias)
    _check_forward(x, cuda_device, kind, k, bias, renorm=True)


def test_ties_go_to_the_lowest_index(cuda_device):
    x = torch.zeros(5, 96)
    x[1, 50] = x[1, 70] = 1.0
    x[2] = torch.arange(96).flip(0) // 8
    x[3, ::2] = -INF
    for kind in ("softmax", "sigmoid"):
        _check_forward(x, cuda_device, kind, 12)
        _check_forward(x, cuda_device, kind, 12, groups=12, topk_groups=3)


@pytest.mark.parametrize("E,k,groups", [(256, 8, 1), (256, 8, 8), (128, 4, 1), (64, 4, 1), (64, 8, 4),
                                        (32, 32, 1), (200, 3, 5)])
def test_rows_of_all_kinds_side_by_side(cuda_device, E, k, groups):
    """Neighbouring tokens, which may share a warp, with nothing in common: all logits equal (more
    ties than are gathered), ordinary, a few experts only, none."""
    x = _logits(E, 41, dict(E=E, kind="sigmoid", groups=groups), torch.float32)
    x[::4] = 0.25
    x[1::4, 3:] = -INF
    x[3::8] = -INF
    for kind in ("softmax", "sigmoid"):
        _check_forward(x, cuda_device, kind, k, groups=groups, topk_groups=max(1, groups // 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_odd_addresses(cuda_device, dtype):
    """Logits as columns of a wider matrix, from an odd element on."""
    x = _logits(9, 21, dict(E=63, kind="softmax"), dtype)
    wide = torch.full((21, 131), NAN, dtype=dtype, device=cuda_device)
    wide[:, 5:68] = x.to(cuda_device)
    view = wide[:, 5:68]
    ids, _ = _check_forward(x, cuda_device, "softmax", 7, logits=view)
    dw = torch.randn(21, 7, device=cuda_device)
    a = tkq.route_topk_backward(view, ids, dw)
    b = tkq.route_topk_backward(view.contiguous(), ids, dw)
    assert torch.equal(a, b)


def _grad_bound(x, ids, dw, kind, renorm, scale):
    s, live = B.scores(x, kind)
    ok = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(ok, ids, 0).long()
    p = torch.where(ok, s.gather(1, at), 0.0)
    a = torch.where(ok, (dw * scale).abs(), 0.0)
    if renorm:
        total = p.sum(1, keepdim=True)
        safe = torch.where(total > 0, total, 1.0)
        a = torch.where(ok & (total > 0), (a + (a * p / safe).sum(1, keepdim=True)) / safe, 0.0)
    ds = torch.zeros_like(x).scatter_add_(1, at, torch.where(ok, a, 0.0))
    if kind == "sigmoid":
        return ds * s
    return s * (ds + (ds * s).sum(1, keepdim=True))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (19, 7, 7), (33, 60, 4), (50, 257, 16),
                                   (8, 1024, 32), (40, 64, 1)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient(cuda_device, T, E, k, kind, renorm, dtype):
    gen = torch.Generator().manual_seed(T + E)
    x = _logits(T * E, T, dict(E=E, kind=kind), dtype)
    if E > 8:
        x[::4, 2::3] = -INF
        x[1::4] = -INF
        x[2::8, 5] = NAN
    ids, _ = B.route(x.double(), k, kind)
    if k > 2:
        ids[::3, 1] = -1                    # an empty slot, and ids that no expert has
        ids[::5, 2] = E
        ids[::7, 0] = -2 ** 31
    dw = torch.randn(T, k, generator=gen)
    dw[ids < 0] = NAN                       # is not read into the result
    dw[ids >= E] = INF
    ref = B.route_backward(x.double(), ids, dw.double().nan_to_num(), kind, renorm, 1.5)
    got = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device), dw.to(cuda_device),
                                  scores=kind, renormalize=renorm, scale=1.5)
    assert got.dtype == dtype and got.shape == x.shape
    bound = (2 * _spread(x, kind) + 96) * U * _grad_bound(
        x.double(), ids, dw.double().nan_to_num(), kind, renorm, 1.5)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs()
    assert (got.cpu().double() - ref).abs().le(bound + 2.0 ** -126).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_against_differences(cuda_device, kind):
    """The kernel's gradient along a direction and the difference quotient of the 64-bit forward:
    off by the quotient's 1e-7 and by the gradient's own bound."""
    gen = torch.Generator().manual_seed(4)
    x = _logits(8, 6, dict(E=24, kind=kind), torch.float32)
    ids, _ = B.route(x.double(), 5, kind)
    dw = torch.randn(6, 5, generator=gen)
    got = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device), dw.to(cuda_device),
                                  scores=kind).cpu().double()
    bound = (2 * _spread(x, kind) + 96) * U * _grad_bound(x.double(), ids, dw.double(), kind, True, 1.0)

    def f(z):
        return (B.route_weights(z, ids, kind, True, 1.0) * dw).sum()
    for _ in range(4):
        v = torch.randn(6, 24, generator=gen, dtype=torch.float64)
        slope = (f(x.double() + 1e-5 * v) - f(x.double() - 1e-5 * v)) / 2e-5
        assert abs(slope - (got * v).sum()) <= 1e-7 + (bound * v.abs()).sum()


def test_single_expert_renormalised_has_no_gradient(cuda_device):
    x = torch.randn(9, 12)
    ids, _ = B.route(x.double(), 1, "softmax")
    for kind in ("softmax", "sigmoid"):
        d = tkq.route_topk_backward(x.to(cuda_device), ids.to(cuda_device),
                                    torch.randn(9, 1, device=cuda_device), scores=kind)
        assert (d == 0).all()


def test_many_tokens_and_counts_add_up(cuda_device):
    """More tokens than one pass of the grid, twice into the same counts."""
    T, E, k = 50001, 96, 6
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn(T, E, generator=gen) * 2).bfloat16().to(cuda_device)
    counts = torch.zeros(E, dtype=torch.int32, device=cuda_device)
    ids, w = tkq.route_topk(x, k, counts=counts)
    tkq.route_topk(x, k, counts=counts)
    order = x.float().sort(dim=1, descending=True, stable=True)      # softmax keeps the order
    assert torch.equal(ids.long(), order.indices[:, :k])
    ref = torch.softmax(order.values[:, :k].double(), 1)
    assert (w.double() - ref).abs().le((2 * 20 + 64) * U * ref).all()
    assert torch.equal(counts.long(), 2 * torch.bincount(ids.flatten().long(), minlength=E))


def test_offsets_beyond_32_bits(cuda_device):
    T, E, k = 2 ** 21 + 70, 1024, 4
    x = torch.full((T, E), -1.0, dtype=torch.bfloat16, device=cuda_device)
    tail = _logits(3, 64, dict(E=E, kind="sigmoid"), torch.bfloat16).to(cuda_device)
    x[-64:] = tail
    ids, w = tkq.route_topk(x, k, scores="sigmoid")
    a, b = tkq.route_topk(tail, k, scores="sigmoid")
    assert torch.equal(ids[-64:], a) and torch.equal(w[-64:], b)
    dw = torch.randn(T, k, device=cuda_device)
    d = tkq.route_topk_backward(x, ids, dw, scores="sigmoid")
    assert torch.equal(d[-64:], tkq.route_topk_backward(tail, a, dw[-64:].contiguous(), scores="sigmoid"))


def test_no_tokens(cuda_device):
    x = torch.empty(0, 16, dtype=torch.bfloat16, device=cuda_device)
    ids, w = tkq.route_topk(x, 4)
    assert ids.shape == w.shape == (0, 4)
    assert tkq.route_topk_backward(x, ids, w).shape == (0, 16)
