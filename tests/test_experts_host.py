"""What the experts' entry points refuse, on the host, before anything is launched: status codes of the C
ABI on addresses that are never dereferenced, and the binding's checks of tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

FAKE = 0x7F0000000000
NULL, SHAPE, GROUP, FMT, ALIGN, ALIAS, FLAGS = 1, 2, 3, 4, 5, 8, 9


@pytest.fixture(scope="module")
def lib():
    from fp8_activation_quantization_gb300 import _build
    _build.build()
    return tkq.load_library()


def at(mb, off=0):
    return ctypes.c_void_p(FAKE + (mb << 20) + off)


def _call(fn, good, **changes):
    """The call with the named arguments of `good` changed."""
    assert set(changes) <= set(good)
    return fn(*{**good, **changes}.values(), None)


@pytest.mark.parametrize("T,k,E,align,rows", [
    (0, 8, 256, 128, 0), (1, 1, 1, 1, 1), (1, 8, 256, 128, 1024), (4, 8, 256, 1, 32), (100, 2, 7, 16, 304),
    (8192, 8, 64, 128, 65536 + 63 * 128), (5, 3, 1024, 1024, 15 * 1024), (-1, 8, 8, 1, -1), (1, 0, 8, 1, -1),
    (1, 33, 64, 1, -1), (1, 8, 0, 1, -1), (1, 8, 1025, 1, -1), (1, 8, 8, 0, -1), (1, 8, 8, 1025, -1),
    (2 ** 30, 2, 8, 1, -1)])
def test_rows_needed(lib, T, k, E, align, rows):
    assert lib.tkq_expert_rows(T, k, E, align) == rows
    if rows >= 0 and T:  # the most rows that any choice of experts needs
        worst = min(E, T * k) - 1
        last = T * k - worst
        assert worst * align + -(-last // align) * align <= rows


ORDER = dict(ids=at(0), slots=at(1), rows=at(2), offsets=at(3), T=4, k=8, E=64, align=16, R=32 * 16)


@pytest.mark.parametrize("changes,expected", [
    (dict(ids=None), NULL), (dict(slots=None), NULL), (dict(rows=None), NULL), (dict(offsets=None), NULL),
    (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(align=0), SHAPE), (dict(align=2000), SHAPE), (dict(R=511), SHAPE), (dict(R=-1), SHAPE),
    (dict(R=2 ** 31), SHAPE), (dict(T=2 ** 30), SHAPE), (dict(ids=at(0, 2)), ALIGN), (dict(offsets=at(3, 1)), ALIGN),
    (dict(slots=at(0)), ALIAS), (dict(rows=at(1, 64)), ALIAS), (dict(offsets=at(2, 2044)), ALIAS)])
def test_order_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_order, ORDER, **changes) == expected


GATHER = dict(x=at(0), x_sf=None, slots=at(1), rows=at(2), offsets=at(3), weights=at(4), out=at(5), out_sf=at(6),
              row_weights=at(7), T=4, C=256, group=128, k=8, E=64, R=512, form=1, fmt=0)


@pytest.mark.parametrize("changes,expected", [
    (dict(x=None), NULL), (dict(slots=None), NULL), (dict(rows=None), NULL), (dict(offsets=None), NULL),
    (dict(out=None), NULL), (dict(out_sf=None), NULL), (dict(weights=None), NULL), (dict(row_weights=None), NULL),
    (dict(x_sf=at(8)), NULL), (dict(form=2), NULL), (dict(form=0), NULL), (dict(form=3), FLAGS), (dict(fmt=2), FMT),
    (dict(group=64), GROUP), (dict(C=200), SHAPE), (dict(C=0), SHAPE), (dict(C=2 ** 21), SHAPE), (dict(T=-1), SHAPE),
    (dict(k=40), SHAPE), (dict(E=0), SHAPE), (dict(R=-1), SHAPE), (dict(x=at(0, 8)), ALIGN), (dict(out=at(5, 4)), ALIGN),
    (dict(out_sf=at(6, 2)), ALIGN), (dict(out=at(0)), ALIAS), (dict(row_weights=at(4)), ALIAS),
    (dict(form=0, out_sf=None, out=at(5, 16)), ALIGN),  # bf16 rows go out in sectors of 32 bytes
    (dict(out_sf=at(5, 1024)), ALIAS), (dict(T=0, x=None), 0), (dict(R=0, out=None), 0)])
def test_gather_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_gather, GATHER, **changes) == expected


REDUCE = dict(y=at(0), slots=at(1), weights=at(2), row_values=at(3), out=at(4), values=at(5), T=4, C=256, group=128, k=8,
              R=512, dtype=1)


@pytest.mark.parametrize("changes,expected", [
    (dict(y=None), NULL), (dict(slots=None), NULL), (dict(out=None), NULL), (dict(values=None), NULL),
    (dict(row_values=None), NULL), (dict(dtype=2), FMT), (dict(group=32), GROUP), (dict(C=100), SHAPE), (dict(T=-2), SHAPE),
    (dict(k=0), SHAPE), (dict(R=2 ** 31), SHAPE), (dict(y=at(0, 2)), ALIGN), (dict(out=at(4, 8)), ALIGN),
    (dict(out=at(0, 4096)), ALIAS), (dict(values=at(2)), ALIAS), (dict(values=at(4, 512)), ALIAS), (dict(T=0, y=None), 0)])
def test_reduce_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_reduce, REDUCE, **changes) == expected


REDUCE_B = dict(dout=at(0), y=at(1), slots=at(2), rows=at(3), offsets=at(4), weights=at(5), dy=at(6), dy_sf=at(7),
                dweights=at(8), T=4, C=256, group=128, k=8, E=64, R=512, form=1, fmt=0)


@pytest.mark.parametrize("changes,expected", [
    (dict(dout=None), NULL), (dict(y=None), NULL), (dict(slots=None), NULL), (dict(rows=None), NULL),
    (dict(offsets=None), NULL), (dict(weights=None), NULL), (dict(dy=None), NULL), (dict(dy_sf=None), NULL),
    (dict(dweights=None), NULL), (dict(form=0), NULL), (dict(form=2), FLAGS), (dict(fmt=7), FMT), (dict(group=1), GROUP),
    (dict(C=129), SHAPE), (dict(E=2000), SHAPE), (dict(dy=at(6, 8)), ALIGN), (dict(dweights=at(8, 2)), ALIGN),
    (dict(dy=at(1)), ALIAS), (dict(dweights=at(5)), ALIAS), (dict(T=0, dout=None), 0)])
def test_reduce_backward_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_reduce_backward, REDUCE_B, **changes) == expected


PRODUCT = dict(a=at(0), a_sf=at(1), w=at(2), w_sf=at(3), offsets=at(4), out=at(5), R=512, E=4, N=256, K=256, group=128,
               fmt_a=0, fmt_w=1)


@pytest.mark.parametrize("changes,expected", [
    *((dict([(n, None)]), NULL) for n in ("a", "a_sf", "w", "w_sf", "offsets", "out")), (dict(R=-1), SHAPE),
    (dict(R=2 ** 31 - 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(N=100), SHAPE), (dict(N=0), SHAPE),
    (dict(K=64), SHAPE), (dict(K=2 ** 21), SHAPE), (dict(E=1024, N=2 ** 21), SHAPE), (dict(E=1024, N=2 ** 20, K=2 ** 20), SHAPE),
    (dict(group=64), GROUP), (dict(fmt_a=2), FMT), (dict(fmt_w=-1), FMT), (dict(a=at(0, 8)), ALIGN), (dict(w=at(2, 4)), ALIGN),
    (dict(out=at(5, 2)), ALIGN), (dict(out=at(5, 16)), ALIGN), (dict(a_sf=at(1, 2)), ALIGN),
    (dict(out=at(0, 131072 - 32)), ALIAS),
    (dict(out=at(4)), ALIAS), (dict(R=0, a=None), 0)])
def test_product_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_product, PRODUCT, **changes) == expected


GRAD = dict(dy_t=at(0), dy_sf=at(1), x_t=at(2), x_sf=at(3), offsets=at(4), dw=at(5), R=512, E=4, N=256, K=256, group=128,
            fmt_dy=1, fmt_x=0, dtype=0)


@pytest.mark.parametrize("changes,expected", [
    *((dict([(n, None)]), NULL) for n in ("dy_t", "dy_sf", "x_t", "x_sf", "offsets", "dw")), (dict(R=100), SHAPE),
    (dict(R=-128), SHAPE), (dict(E=0), SHAPE), (dict(N=130), SHAPE), (dict(K=0), SHAPE), (dict(group=32), GROUP),
    (dict(fmt_dy=2), FMT), (dict(fmt_x=3), FMT), (dict(dtype=2), FMT), (dict(dy_t=at(0, 4)), ALIGN), (dict(dw=at(5, 8)), ALIGN),
    (dict(dw=at(5, 16)), ALIGN), (dict(dw=at(5, 16), dtype=1), ALIGN),
    (dict(dw=at(2)), ALIAS), (dict(R=0, dy_t=None, offsets=None), NULL)])
def test_weight_grad_refusals(lib, changes, expected):
    assert _call(lib.tkq_expert_weight_grad, GRAD, **changes) == expected


W4 = dict(x=at(0), x_sf=at(1), w=at(2), w_sf=at(3), ids=at(4), out=at(5), T=4, k=2, rows=4, E=4, N=256, K=256, group=128,
          w_group=32, fmt=0)


@pytest.mark.parametrize("changes,expected", [
    *((dict([(n, None)]), NULL) for n in ("x", "x_sf", "w", "w_sf", "out")), (dict(ids=None), SHAPE),
    (dict(ids=None, k=1, E=2), SHAPE), (dict(rows=5), SHAPE), (dict(T=1024), SHAPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE),
    (dict(N=64), SHAPE), (dict(K=192), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(group=64), GROUP),
    (dict(w_group=64), GROUP), (dict(fmt=4), FMT), (dict(x=at(0, 8)), ALIGN), (dict(w=at(2, 8)), ALIGN),
    (dict(out=at(5, 8)), ALIGN), (dict(w_sf=at(3, 2)), ALIGN), (dict(out=at(2)), ALIAS), (dict(T=0, rows=0, x=None), 0)])
def test_w4_product_refusals(lib, changes, expected):
    assert _call(lib.tkq_w4_product, W4, **changes) == expected


W4C = dict(w=at(0), codes=at(1), sf=at(2), N=16, K=256, w_group=32)


@pytest.mark.parametrize("changes,expected", [
    (dict(w=None), NULL), (dict(codes=None), NULL), (dict(sf=None), NULL), (dict(N=-1), SHAPE), (dict(K=100), SHAPE),
    (dict(K=0), SHAPE), (dict(w_group=16), GROUP), (dict(w=at(0, 8)), ALIGN), (dict(codes=at(1, 2)), ALIGN),
    (dict(codes=at(0)), ALIAS), (dict(N=0, w=None), 0)])
def test_w4_cast_refusals(lib, changes, expected):
    assert _call(lib.tkq_w4_cast, W4C, **changes) == expected


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    order = tkq.ExpertOrder(i32(4, 2), i32(16), i32(5))
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    f8 = lambda *s: torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: tkq.expert_order(i32(4, 2), 8), lambda: tkq.expert_order(None, 8), lambda: tkq.expert_gather(x, order),
                 lambda: tkq.expert_gather(f8(4, 256), order, x_sf=torch.zeros(4, 2)), lambda: tkq.expert_reduce(x, order),
                 lambda: tkq.expert_reduce_backward(x, x, order, torch.zeros(4, 2)),
                 lambda: tkq.expert_product(f8(4, 256), torch.zeros(4, 2), f8(4, 128, 256), torch.zeros(4, 1, 2), i32(5)),
                 lambda: tkq.expert_weight_grad(f8(128, 128), torch.zeros(128, 1), f8(128, 128), torch.zeros(128, 1), i32(5)),
                 lambda: tkq.w4_product(f8(4, 256), torch.zeros(4, 2), torch.zeros(128, 128, dtype=torch.uint8),
                                        torch.zeros(128, 8, dtype=torch.uint8)),
                 lambda: tkq.w4_cast(x)):
        with pytest.raises(TypeError):
            call()


def test_binding_checks_of_an_order():
    dev = torch.device("cpu")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = (i32(4, 2), i32(16), i32(5))
    assert tkq._check_order(good, dev) == (4, 2, 16, 4) and tkq._check_order(tkq.ExpertOrder(*good), dev, 4) == (4, 2, 16, 4)
    for bad in (None, good[:2], (i32(8), *good[1:]), (good[0], i32(2, 8), good[2]), (*good[:2], i32(1)),
                (good[0].long(), *good[1:]), (good[0], good[1].float(), good[2]), (*good[:2], i32(10)[::2])):
        with pytest.raises(TypeError):
            tkq._check_order(bad, dev)
    with pytest.raises(ValueError):
        tkq._check_order(good, dev, 5)


def test_the_formulas_agree_with_one_another():
    """The 64-bit formulas themselves: places round trip, sums, and the products on whole numbers."""
    g = torch.Generator().manual_seed(0)
    ids = torch.rand(20, 9, generator=g).topk(3, 1).indices.int()
    ids[3] = -1
    slots, rows, offsets = experts64.order(ids, 9, 16, 400)
    live = rows >= 0
    assert int(live.sum()) == 57 and torch.equal(slots.flatten()[rows[live].long()].long(), live.nonzero().flatten())
    assert bool((offsets % 16 == 0).all()) and int(offsets[-1]) <= 400
    y, w = torch.randn(400, 128, generator=g), torch.rand(20, 3, generator=g)
    out, _ = experts64.reduce(y, slots, w)
    want = sum(w[:, j:j + 1].double() * y.double()[slots[:, j].clamp_min(0).long()] * (slots[:, j:j + 1] >= 0) for j in range(3))
    assert torch.allclose(out, want, atol=1e-12)
    d = torch.randn(20, 128, generator=g)
    y2, w2 = y.double().requires_grad_(), w.double().requires_grad_()
    at = slots.clamp_min(0).long()
    ((y2[at] * w2.unsqueeze(2) * (slots >= 0).unsqueeze(2)).sum(1) * d.double()).sum().backward()
    dy, dw, _ = experts64.reduce_backward(d, y, slots, w)
    assert torch.allclose(dw, w2.grad, atol=1e-10)
    assert torch.allclose(experts64.spread(dy, slots, 400), y2.grad, atol=1e-12)
    table = experts64.w4_decoded(torch.arange(256, dtype=torch.uint8).view(4, 64), torch.full((4, 4), 128, dtype=torch.uint8))
    assert float(table.abs().max()) == 12.0 and table[0, 2] == 2 * 0.5 and table[0, 3] == 0.0
