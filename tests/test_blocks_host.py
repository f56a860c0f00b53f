"""What the routing, checkpoint and norm entry points refuse, on the host, before anything is
launched: status codes of the C ABI on addresses that are never dereferenced, and the binding's
checks of tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq

FAKE = 0x7F0000000000
NULL, SHAPE, GROUP, FMT, ALIGN, ALIAS, FLAGS, VALUE = 1, 2, 3, 4, 5, 8, 9, 10
INF = float("inf")


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


ROUTE = dict(logits=at(0), bias=at(1), ids=at(2), weights=at(3), counts=at(4), T=4, E=64, ld=64,
             dtype=0, k=8, groups=4, topk_groups=2, top=2, flags=3, scale=1.0)


@pytest.mark.parametrize("changes,expected", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(ld=63), SHAPE),
    (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=4, k=8), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=33, E=66, ld=66), SHAPE), (dict(groups=5), SHAPE), (dict(topk_groups=0), SHAPE),
    (dict(topk_groups=5), SHAPE), (dict(top=0), VALUE), (dict(top=3), VALUE),
    (dict(dtype=2), FMT), (dict(flags=4), FLAGS), (dict(scale=INF), VALUE),
    (dict(scale=float("nan")), VALUE), (dict(logits=at(0, 2)), ALIGN), (dict(bias=at(1, 2)), ALIGN),
    (dict(ids=at(2, 1)), ALIGN), (dict(counts=at(4, 2)), ALIGN), (dict(ids=at(0, 512)), ALIAS),
    (dict(weights=at(2, 64)), ALIAS), (dict(counts=at(3, 124)), ALIAS), (dict(T=0, logits=None), 0),
    (dict(ids=at(0, 1280), ld=512), ALIAS),       # inside the strided rows
])
def test_route_refusals(lib, changes, expected):
    assert _call(lib.tkq_route_topk, ROUTE, **changes) == expected


ROUTE_B = dict(logits=at(0), ids=at(1), dweights=at(2), dlogits=at(3), T=4, E=64, ld=64, dtype=1,
               k=8, flags=3, scale=1.0)


@pytest.mark.parametrize("changes,expected", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(dweights=None), NULL),
    (dict(dlogits=None), NULL), (dict(k=33), SHAPE), (dict(ld=8), SHAPE), (dict(flags=8), FLAGS),
    (dict(dtype=5), FMT), (dict(scale=-INF), VALUE), (dict(dlogits=at(3, 1)), ALIGN),
    (dict(dlogits=at(0)), ALIAS), (dict(T=0), 0)])
def test_route_backward_refusals(lib, changes, expected):
    assert _call(lib.tkq_route_topk_backward, ROUTE_B, **changes) == expected


SAVE = dict(x=at(0), w=at(1), out=at(2), sf=at(3), ckpt=at(4), ckpt_sf=at(5), T=4, H=256, group=128,
            fmt=0, ckpt_fmt=1, sf_flags=0)


@pytest.mark.parametrize("changes,expected", [
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(sf=None), NULL), (dict(ckpt=None), NULL),
    (dict(ckpt_sf=None), NULL), (dict(H=200), SHAPE), (dict(T=-1), SHAPE), (dict(group=64), GROUP),
    (dict(fmt=2), FMT), (dict(ckpt_fmt=2), FMT), (dict(sf_flags=16), FLAGS),
    (dict(ckpt=at(4, 8)), ALIGN), (dict(sf=at(3, 4), sf_flags=4), ALIGN), (dict(w=at(1, 1)), ALIGN),
    (dict(ckpt=at(0)), ALIAS), (dict(ckpt=at(2, 512)), ALIAS), (dict(ckpt_sf=at(3, 16)), ALIAS),
    (dict(w=at(2)), ALIAS), (dict(T=0, x=None), 0)])
def test_save_refusals(lib, changes, expected):
    assert _call(lib.tkq_swiglu_cast_checkpoint, SAVE, **changes) == expected


RESTORE = dict(ckpt=at(0), ckpt_sf=at(1), dy=at(2), w=at(3), dx=at(4), dx_sf=at(5), y=at(6),
               dw=at(7), T=4, H=256, group=128, ckpt_fmt=0, fmt=0, sf_flags=0)


@pytest.mark.parametrize("changes,expected", [
    (dict(ckpt=None), NULL), (dict(ckpt_sf=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL),
    (dict(dx_sf=None), NULL), (dict(H=130), SHAPE), (dict(group=32), GROUP), (dict(fmt=2), FMT),
    (dict(ckpt_fmt=-1), FMT), (dict(sf_flags=32), FLAGS), (dict(dy=at(2, 8)), ALIGN),
    (dict(y=at(6, 2)), ALIGN), (dict(dw=at(7, 2)), ALIGN), (dict(dx=at(0, 16)), ALIAS),
    (dict(y=at(4, 1024)), ALIAS), (dict(dw=at(5)), ALIAS), (dict(T=0, dy=None), 0)])
def test_restore_refusals(lib, changes, expected):
    assert _call(lib.tkq_swiglu_checkpoint_backward_cast, RESTORE, **changes) == expected
    if not {"dx_sf", "fmt", "sf_flags"} & set(changes) and expected != ALIAS:
        good = {k: v for k, v in RESTORE.items() if k not in ("dx_sf", "fmt", "sf_flags")}
        assert _call(lib.tkq_swiglu_checkpoint_backward, good, **changes) == expected


NORM = dict(r=at(0), h=at(1), w_post=at(2), gate=at(3), w_pre=at(4), r_out=at(5), out=at(6), sf=at(7),
            x=at(8), p=at(9), q=at(10), T=4, C=256, group=128, fmt=0, sf_flags=0, flags=3, a=1.0,
            eps=1e-6)


@pytest.mark.parametrize("changes,expected", [
    (dict(r=None), NULL), (dict(r_out=None), NULL), (dict(sf=None), NULL), (dict(out=None), NULL),
    (dict(out=None, sf=None, x=None), NULL), (dict(C=200), SHAPE), (dict(C=16512), SHAPE),
    (dict(T=-2), SHAPE), (dict(group=1), GROUP), (dict(fmt=3), FMT), (dict(sf_flags=64), FLAGS),
    (dict(flags=8), FLAGS), (dict(h=None), FLAGS), (dict(flags=2), FLAGS), (dict(flags=1), FLAGS),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(a=INF), VALUE),
    (dict(gate=at(3, 2)), ALIGN), (dict(w_pre=at(4, 4)), ALIGN), (dict(p=at(9, 1)), ALIGN),
    (dict(r_out=at(0)), ALIAS), (dict(x=at(6)), ALIAS), (dict(q=at(9, 8)), ALIAS),
    (dict(T=0, r=None), 0)])
def test_norm_refusals(lib, changes, expected):
    assert _call(lib.tkq_residual_norm_cast, NORM, **changes) == expected


NORM_B = dict(dr=at(0), dx=at(1), r=at(2), h=at(3), w_post=at(4), gate=at(5), w_pre=at(6), p=at(7),
              q=at(8), dr_out=at(9), dh=at(10), dgate=at(11), dw_post=at(12), dw_pre=at(13),
              work=at(64), T=4, C=256, flags=3, a=1.0)


@pytest.mark.parametrize("changes,expected", [
    (dict(dx=None), NULL), (dict(r=None), NULL), (dict(q=None), NULL), (dict(p=None), NULL),
    (dict(dr_out=None), NULL), (dict(dh=None), NULL), (dict(dgate=None), NULL), (dict(work=None), NULL),
    (dict(C=100), SHAPE), (dict(C=32768), SHAPE), (dict(flags=16), FLAGS), (dict(flags=1), FLAGS),
    (dict(h=None), FLAGS), (dict(gate=None), FLAGS), (dict(a=float("nan")), VALUE),
    (dict(dr=at(0, 2)), ALIGN), (dict(work=at(64, 4)), ALIGN), (dict(dr_out=at(0)), ALIAS),
    (dict(dgate=at(5)), ALIAS), (dict(dw_pre=at(64, 16)), ALIAS), (dict(T=0, dr=None), 0)])
def test_norm_backward_refusals(lib, changes, expected):
    assert _call(lib.tkq_residual_norm_backward, NORM_B, **changes) == expected


def test_workspace_sizes(lib):
    assert lib.tkq_residual_norm_workspace(0, 256) == 0
    assert lib.tkq_residual_norm_workspace(1, 256) >= 2 * 256 * 4
    assert lib.tkq_residual_norm_workspace(4, 200) == -1
    assert lib.tkq_residual_norm_workspace(-1, 256) == -1


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tkq.route_topk(x, 4)
    with pytest.raises(TypeError):
        tkq.route_topk_backward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(TypeError):
        tkq.swiglu_forward_cast_and_checkpoint(x)
    with pytest.raises(TypeError):
        tkq.swiglu_backward_from_checkpoint(x, x, x)
    with pytest.raises(TypeError):
        tkq.residual_norm_and_cast(x)
    with pytest.raises(TypeError):
        tkq.residual_norm_backward(x, x)


@pytest.mark.parametrize("bad,err", [
    (lambda: torch.zeros(4, 8), TypeError),                                # another type
    (lambda: torch.zeros(8, 4, dtype=torch.bfloat16).t(), TypeError),      # not contiguous
    (lambda: torch.zeros(4, 9, dtype=torch.bfloat16), ValueError),         # another shape
    (lambda: None, TypeError)])
def test_binding_checks_operands(bad, err):
    with pytest.raises(err):
        tkq._check_like(bad(), "h", (4, 8), (torch.bfloat16,), torch.device("cpu"))
