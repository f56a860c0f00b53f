"""The routing, checkpoint and norm kernels over more rows than one pass of their grids, and in the
instances that small inputs do not reach, against the 64-bit formulas.

TKQ_NUM_SMS = 1 sizes the grids as for one SM, so that a few hundred rows take every CTA through more
rows than it keeps in flight, and the norms' forward takes two rows at a time from four rows on.  The
checks and their bounds are those of test_gpu_residual_norm, test_gpu_swiglu_ckpt and test_gpu_route,
which do not depend on how rows are spread."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import test_gpu_residual_norm as norms
from tests import test_gpu_route as route
from tests import test_gpu_swiglu_ckpt as ckpt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    tkq.load_library()
    yield


@pytest.fixture
def one_sm(monkeypatch):
    monkeypatch.setenv("TKQ_NUM_SMS", "1")


# a width of each way to hold a row: less than a warp of vectors, whole and ragged numbers of warps, one
# vector a thread and two, whole and ragged; rows 1, 2, 3 more than a multiple of four
FORWARD = [(203, 128), (197, 640), (198, 1024), (67, 4096), (41, 4224), (38, 6016), (37, 7168), (39, 7296),
           (38, 8192), (5, 4224), (4, 128)]


@pytest.mark.parametrize("T,C", FORWARD)
@pytest.mark.parametrize("f32", [False, True])
def test_norm_forward(cuda_device, one_sm, T, C, f32):
    norms.test_forward(cuda_device, T, C, f32, True, True, True, True)
    norms.test_forward(cuda_device, T, C, f32, False, False, True, False)
    norms.test_norm_before_the_first_block(cuda_device, T, C, f32)


@pytest.mark.parametrize("T,C,f32", [(609, 640, False), (610, 4224, True), (1301, 1024, True),
                                     (1302, 384, False), (611, 7168, False)])
def test_norm_forward_of_a_batch(cuda_device, T, C, f32):
    """The same without the override: as many rows as make the device take two at a time."""
    norms.test_forward(cuda_device, T, C, f32, True, True, True, True)


@pytest.mark.parametrize("T,C", FORWARD)
def test_packed_column_major_scales(cuda_device, one_sm, T, C):
    """One byte a scale in columns: the bytes of the row-major form, zeros in the padding rows and words."""
    _, dev = norms._inputs(T, T, C, False, True, True, True, cuda_device)
    _, a, row, _, _, _ = tkq.residual_norm_and_cast(**dev, use_packed_ue8m0=True)
    _, b, col, _, _, _ = tkq.residual_norm_and_cast(**dev, use_packed_ue8m0=True,
                                                    use_tma_aligned_col_major_sf=True)
    assert torch.equal(norms._bytes(a), norms._bytes(b))
    assert torch.equal(col[:, :T].t(), row) and (col[:, T:] == 0).all()


@pytest.mark.parametrize("T,C", [(203, 128), (197, 640), (67, 2176), (67, 4096), (19, 4224), (19, 6016),
                                 (17, 7168), (18, 7296), (17, 8192), (13, 8320), (9, 16384)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("post,gated,w_post,w_pre,pre,with_dr", [
    (True, True, True, True, True, True), (True, False, True, True, True, True),
    (False, True, True, True, True, False)])
def test_norm_backward(cuda_device, one_sm, T, C, f32, post, gated, w_post, w_pre, pre, with_dr):
    norms.test_backward(cuda_device, T, C, f32, post, gated, w_post, w_pre, pre, with_dr)


@pytest.mark.parametrize("T,H", [(403, 128), (201, 256), (203, 384), (130, 640), (101, 1408), (70, 2048)])
@pytest.mark.parametrize("ckpt_fmt", ["e4m3", "e5m2"])
def test_checkpoint(cuda_device, one_sm, T, H, ckpt_fmt):
    for weighted in (False, True):
        ckpt.test_forward_is_the_two_casts(cuda_device, T, H, weighted, "e4m3", ckpt_fmt)
        ckpt.test_backward(cuda_device, T, H, weighted, ckpt_fmt)


# 401 rows of 1024 sigmoids without a pair too near to order are not to be had
@pytest.mark.parametrize("E,k,groups,kind", [
    (256, 8, 8, "softmax"), (256, 8, 8, "sigmoid"), (256, 8, 1, "softmax"), (256, 8, 1, "sigmoid"),
    (60, 4, 1, "softmax"), (60, 4, 1, "sigmoid"), (36, 6, 3, "softmax"), (36, 6, 3, "sigmoid"),
    (1024, 32, 1, "softmax")])
def test_routing(cuda_device, one_sm, E, k, groups, kind):
    T = 401
    gen = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=gen) * (0.05 if kind == "sigmoid" else 0.5 / E)
    for dtype, b in ((torch.float32, bias), (torch.bfloat16, None)):
        x = route._logits(E + k, T, dict(E=E, kind=kind, groups=groups), dtype, bias=b, mask=route._holes)
        route._check_forward(x, cuda_device, kind, k, b, groups=groups, topk_groups=max(1, groups // 2))
    for renorm in (False, True):
        route.test_gradient(cuda_device, T, E, k, kind, renorm, torch.float32)


def _counted_calls(device):
    gen = torch.Generator().manual_seed(1)
    calls = []
    for T, E, k, groups in [(1, 256, 8, 8), (37, 60, 4, 1), (130, 1024, 32, 32), (5000, 96, 6, 1)]:
        x = torch.randn(T, E, generator=gen).to(device)
        counts = torch.zeros(E, dtype=torch.int32, device=device)

        def call(x=x, k=k, groups=groups, counts=counts):
            counts.zero_()
            ids, _ = tkq.route_topk(x, k, "sigmoid", num_groups=groups, topk_groups=max(1, groups // 2),
                                    counts=counts)
            return ids, counts
        calls.append(call)
    return calls


def _check_counts(ids, counts):
    assert torch.equal(counts.long(), torch.bincount(ids[ids >= 0].long(), minlength=len(counts)))


def test_counts_of_the_checked_build(cuda_device):
    from fp8_activation_quantization_gb300 import _build
    _build.build(checked=True)
    for call in _counted_calls(cuda_device):
        ids, ref = (t.clone() for t in call())
        _check_counts(ids, ref)
        with tkq.use_checked_library():
            got, counts = (t.clone() for t in call())
        assert torch.equal(got, ids) and torch.equal(counts, ref)


def test_counts_of_graph_replays(cuda_device):
    for call in _counted_calls(cuda_device):
        ref = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ids, counts = call()
        for _ in range(3):
            ids.zero_()
            counts.fill_(-7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(ids, ref[0]) and torch.equal(counts, ref[1])
            _check_counts(ids, counts)
