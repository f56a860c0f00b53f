"""Products with 4-bit weights and the cast that makes them, against their 64-bit formulas.

The cast is compared exactly.  A product's bound, with u = 2^-24 and b = 2^-8 (half steps of binary32 and
bf16): products of codes are exact; the tensor core adds 16 of them and the accumulator at a time, which
may be cut off and aligned to the largest (17 terms, each off by at most 2 u of a value no larger than the
sum of magnitudes), twice a group of 32; a group's scale, its sum's product with it and the additions of
groups, blocks and, where warps share rows, of up to 16 parts are rounded once each: (4 x 2 x 17 x 2 + 4 +
4 + K / 128 + 16) u of the sum of magnitudes, and the result's b."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def weights(shape, group, g):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, generator=g)
    if group == 32:
        return codes, torch.randint(100, 150, (*shape[:-1], shape[-1] // 32), dtype=torch.uint8, generator=g)
    return codes, torch.randn(*shape[:-1], shape[-1] // 128, generator=g)


def check(got, ref, size, K):
    bound = (4 * 2 * 17 * 2 + 8 + K // 128 + 16) * U * size + B * (1 + B) * ref.abs()
    off = (got.cpu().double() - ref).abs() > bound + 1e-38
    assert not bool(off.any()), (int(off.sum()), off.nonzero()[:4].tolist())


def codes(rows, K, fmt, g, dev):
    x = torch.randn(rows, K, generator=g) * torch.rand(rows, 1, generator=g).mul(6).exp()
    return tkq.per_token_cast(x.bfloat16().to(dev), fmt)


@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (1, 4096, 2048), (3, 256, 384), (8, 128, 4096), (9, 640, 256),
                                   (16, 384, 1408), (17, 128, 640), (64, 256, 896), (100, 128, 128), (1024, 128, 256)])
@pytest.mark.parametrize("group,fmt", [(32, "e4m3"), (128, "e4m3"), (32, "e5m2"), (128, "e5m2")])
def test_one_matrix(cuda_device, T, N, K, group, fmt):
    g = gen(T + N + K)
    x, xs = codes(T, K, fmt, g, cuda_device)
    w, ws = weights((N, K), group, g)
    got = tkq.w4_product(x, xs, w.to(cuda_device), ws.to(cuda_device))
    ref, size = experts64.w4_product(x.cpu().float(), xs.cpu(), w, ws, None, False)
    check(got, ref, size, K)


@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 16, 256, 256), (1, 1, 1, 128, 128), (4, 4, 60, 128, 512), (9, 2, 3, 384, 128),
                                       (48, 6, 7, 128, 384), (33, 1, 1024, 128, 128), (32, 32, 40, 128, 256)])
@pytest.mark.parametrize("group,each", [(32, False), (32, True), (128, False), (128, True)])
def test_experts(cuda_device, T, k, E, N, K, group, each):
    g = gen(T + N + K + E)
    x, xs = codes(T * k if each else T, K, "e4m3", g, cuda_device)
    w, ws = weights((E, N, K), group, g)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=g)  # some of them twice
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    if T > 3:
        ids[2, 0], ids[3, 0] = E, 2 ** 31 - 1
    out = torch.full((T * k, N), 7.0, dtype=BF16, device=cuda_device)
    got = tkq.w4_product(x, xs, w.to(cuda_device), ws.to(cuda_device), ids.to(cuda_device), out=out)
    ref, size = experts64.w4_product(x.cpu().float(), xs.cpu(), w, ws, ids, each)
    check(got, ref, size, K)
    assert got is out
    assert torch.equal(tkq.w4_product(x, xs, w.to(cuda_device), ws.to(cuda_device), ids.to(cuda_device)), got)


def test_whole_numbers_are_exact(cuda_device):
    g = gen(2)
    T, N, K = 13, 256, 640
    x = torch.randint(-2, 3, (T, K), generator=g).float()
    xs = torch.randint(-2, 3, (T, K // 128), generator=g).float().exp2()
    w, ws = weights((N, K), 32, g)
    ws = ws // 25 + 123
    got = tkq.w4_product(x.to(torch.float8_e4m3fn).to(cuda_device), xs.to(cuda_device), w.to(cuda_device), ws.to(cuda_device))
    ref, _ = experts64.w4_product(x, xs, w, ws, None, False)
    assert torch.equal(got.cpu(), ref.to(BF16))


def test_every_code_and_scale(cuda_device):
    """One nonzero code a row picks each 4-bit code, and each byte's scale, out exactly."""
    K, N = 128, 256
    w = torch.zeros(N, K // 2, dtype=torch.uint8)
    w[:, 0] = torch.arange(256, dtype=torch.uint8)
    x = torch.zeros(2, K)
    x[0, 0] = x[1, 1] = 1.0
    ws = torch.full((N, K // 32), 127, dtype=torch.uint8)
    args = lambda *v: [t.to(cuda_device) for t in v]
    xs = torch.ones(2, 1)
    got = tkq.w4_product(*args(x.to(torch.float8_e4m3fn), xs, w, ws)).cpu().double()
    table = torch.from_numpy(experts64.E2M1)
    assert torch.equal(got[0], table[torch.arange(256) % 16].abs() * torch.sign(table[torch.arange(256) % 16]))
    assert torch.equal(got[1], table[torch.arange(256) // 16])
    w[:, 0] = 2  # 1.0
    ws[:, 0] = torch.arange(256, dtype=torch.uint8)
    ws[255, 0] = 127
    got = tkq.w4_product(*args(x.to(torch.float8_e4m3fn), xs, w, ws)).cpu().double()
    ref = torch.exp2(torch.arange(256).double() - 127)
    ref[255] = 1.0
    assert torch.equal(got[0], ref)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (5, 384), (300, 2048)])
def test_cast(cuda_device, group, N, K):
    g = gen(N + K)
    w = (torch.randn(N, K, generator=g) * torch.rand(N, 1, generator=g).mul(40).sub(20).exp()).bfloat16()
    w[0, :64] = 0
    w[-1, -1] = 3e38
    codes, sf = tkq.w4_cast(w.to(cuda_device), group)
    v = w.float().view(N, -1, group)
    s = torch.maximum(v.abs().amax(2) / 6, torch.tensor(2.0 ** -126))
    if group == 32:
        m, e = torch.frexp(s)
        e = e - (m == 0.5).int()  # s = 2^e, rounded up
        assert torch.equal(sf.cpu().int(), e + 127)
        s = torch.exp2(e.double()).float()
    else:
        assert torch.equal(sf.cpu(), s)
    q = (v / s.unsqueeze(2)).double().abs().view(N, K)
    size = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6]).double()
    far = (q.unsqueeze(2) - size).abs()
    even = torch.arange(8) % 2 * 1e-9  # ties to the even code
    want = (far + even).argmin(2) + 8 * torch.signbit(w.float()).long()
    c = codes.cpu().long()
    got = torch.stack([c & 15, c >> 4], 2).view(N, K)
    assert torch.equal(got, want)


def test_cast_and_product_together(cuda_device):
    g = gen(4)
    w = torch.randn(3, 256, 512, generator=g).bfloat16().to(cuda_device)
    x, xs = codes(5, 512, "e4m3", g, cuda_device)
    ids = torch.tensor([[0, 2], [1, 1], [2, 0], [-1, 1], [0, 1]], dtype=torch.int32)
    for group in (32, 128):
        q, sf = tkq.w4_cast(w, group)
        assert q.shape == (3, 256, 256) and sf.shape == (3, 256, 512 // group)
        got = tkq.w4_product(x, xs, q, sf, ids.to(cuda_device))
        ref, size = experts64.w4_product(x.cpu().float(), xs.cpu(), q.cpu(), sf.cpu(), ids, False)
        check(got, ref, size, 512)
