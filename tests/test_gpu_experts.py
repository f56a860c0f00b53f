"""Rows by expert and back, and the experts' FP8 products, against their 64-bit formulas.

Bounds, with u = 2^-24 (half a step of binary32), b = 2^-8 (of bf16):
* places, copies and casts are compared exactly (the cast with per_token_cast);
* a sum of k weighted rows: one rounding of each product-and-add, k u of the sum of magnitudes, and the
  result's b;
* dweights: a lane adds 8 products per eight groups, then 5 steps of the warp and 4 of the CTA, each
  rounded once: (8 ceil(G / 8) + 10) u of the sum of magnitudes;
* a product: the tensor core adds 32 exact products and the accumulator at a time, which may be cut
  off instead of rounded and aligned to the largest of them (33 terms, each off by at most a step, 2 u,
  of a value no larger than the sum of magnitudes), four times a group; the scales' product, its product
  with the group's sum and the sum of the groups are rounded once each: (4 x 33 x 2 + 3 + G) u of the
  sum of magnitudes, and the result's b where it is bf16."""
from __future__ import annotations

import pytest
import torch

import fp8_activation_quantization_gb300 as tkq
from tests import experts64

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def ids_of(T, k, E, g, empty=0.1):
    ids = torch.rand(T, E, generator=g).pow(3).topk(k, 1).indices.int()
    ids[torch.rand(T, k, generator=g) < empty] = -1
    return ids


def close(got, ref, bound):
    got = got.cpu().double()
    off = (got - ref).abs() > bound
    assert not bool(off.any()), (int(off.sum()), float((got - ref).abs().max()))


ORDERS = [(1, 1, 1, 1), (1, 8, 256, 1), (4, 8, 256, 128), (33, 2, 7, 16), (1021, 6, 60, 128), (1, 1, 1024, 128),
          (700, 32, 64, 1), (5000, 1, 3, 128), (9001, 8, 60, 5), (64, 3, 4, 1024)]


@pytest.mark.parametrize("T,k,E,align", ORDERS)
def test_order(cuda_device, T, k, E, align):
    ids = ids_of(T, k, E, gen(T + k))
    got = tkq.expert_order(ids.to(cuda_device), E, align)
    for name, a, b in zip(got._fields, got, experts64.order(ids, E, align, got.rows.numel())):
        assert torch.equal(a.cpu(), b), name


@pytest.mark.parametrize("case", ["all empty", "one expert", "ids out of range", "the same expert twice", "no tokens"])
def test_order_of_unusual_choices(cuda_device, case):
    T, k, E = (0 if case == "no tokens" else 130), 4, 9
    ids = {"all empty": torch.full((T, k), -1), "one expert": torch.full((T, k), 8), "no tokens": torch.zeros(T, k),
           "the same expert twice": torch.arange(T).unsqueeze(1) % 3 + torch.zeros(1, k),
           "ids out of range": torch.randint(-2 ** 31, 2 ** 31 - 1, (T, k), generator=gen())}[case].int()
    if case == "ids out of range":
        ids[::3, 1] = 9
        ids[::5, 2] = 3
    got = tkq.expert_order(ids.to(cuda_device), E, 16)
    for name, a, b in zip(got._fields, got, experts64.order(ids, E, 16, got.rows.numel())):
        assert torch.equal(a.cpu(), b), name


def test_order_in_larger_buffers_and_repeated(cuda_device):
    ids = ids_of(3000, 8, 40, gen(1)).to(cuda_device)
    rows = torch.full((40000,), 5, dtype=torch.int32, device=cuda_device)
    a = tkq.expert_order(ids, 40, 128, rows=rows)
    assert a.rows is rows and int((rows >= 0).sum()) == int((ids >= 0).sum()) and int(rows.min()) == -1
    b = tkq.expert_order(ids, 40, 128)
    assert torch.equal(a.rows[:b.rows.numel()], b.rows) and torch.equal(a.slots, b.slots)
    # as many pairs as a small cluster, a full one and several passes of it take
    for T in (512, 513, 2048, 4096, 4097, 40000):
        ids = ids_of(T, 8, 33, gen(T)).to(cuda_device)
        got = tkq.expert_order(ids, 33, 128)
        key = torch.where(ids >= 0, ids, 33).flatten()
        perm = key.argsort(stable=True)[: int((key < 33).sum())]
        assert torch.equal(got.rows[got.rows >= 0].long(), perm)
        assert torch.equal(got.slots.flatten()[perm].long(), (got.rows >= 0).nonzero().flatten())


ROWS = [(1, 1, 1, 128, 1), (4, 8, 256, 7168, 1), (4, 8, 256, 1408, 128), (33, 2, 7, 640, 16), (257, 6, 60, 384, 128),
        (130, 32, 40, 256, 1), (1000, 3, 5, 128, 128), (5, 8, 8, 2048, 3)]


@pytest.mark.parametrize("T,k,E,C,align", ROWS)
@pytest.mark.parametrize("form", ["bf16", "e4m3", "e5m2", "codes"])
def test_gather(cuda_device, T, k, E, C, align, form):
    g = gen(C + T)
    ids = ids_of(T, k, E, g)
    x = torch.randn(T, C, generator=g).bfloat16().to(cuda_device)
    w = torch.rand(T, k, generator=g)
    order = tkq.expert_order(ids.to(cuda_device), E, align)
    R, end = order.rows.numel(), int(order.offsets[-1])
    kw = {}
    sf = None
    if form == "bf16":
        rows = x
        buf = torch.full((R, C), GUARD, dtype=BF16, device=cuda_device)
    else:
        rows, sf = tkq.per_token_cast(x, form if form != "codes" else "e5m2")
        buf = torch.full((R, C), 0x55, dtype=torch.uint8, device=cuda_device)
        kw["out_sf"] = torch.full((R, C // 128), GUARD, device=cuda_device)
    if form == "codes":
        out, out_sf, rw = tkq.expert_gather(rows, order, x_sf=sf, weights=w.to(cuda_device), out=buf, **kw)
    else:
        out, out_sf, rw = tkq.expert_gather(x, order, fmt=None if form == "bf16" else form, weights=w.to(cuda_device),
                                            out=buf, **kw)
    assert out is buf
    pair = order.rows.cpu().long()
    live, behind = pair >= 0, torch.arange(R) >= end
    pad = ~live & ~behind
    bits = lambda v: v.view(torch.uint8 if v.element_size() == 1 else torch.int16).cpu()
    out, rows = bits(out), bits(rows)
    assert torch.equal(out[live], rows[pair[live] // k])
    assert not bool(out[pad].any())
    assert torch.equal(out[behind], bits(torch.full((R, C), GUARD, dtype=BF16) if form == "bf16" else
                                         torch.full((R, C), 0x55, dtype=torch.uint8))[behind])
    rw = rw.cpu()
    assert torch.equal(rw[live], w.flatten()[pair[live]]) and not bool(rw[pad].any())
    if sf is not None:
        out_sf, sf = out_sf.cpu(), sf.cpu()
        assert torch.equal(out_sf[live], sf[pair[live] // k])
        zero = 0.0 if form == "codes" else torch.tensor(1e-4) / {"e4m3": 448.0, "e5m2": 57344.0}[form]
        assert bool((out_sf[pad] == zero).all()) and bool((out_sf[behind] == GUARD).all())


def test_gather_skips_bad_slots(cuda_device):
    order = tkq.expert_order(ids_of(50, 4, 6, gen(), 0).to(cuda_device), 6, 16)
    x = torch.ones(50, 256, dtype=BF16, device=cuda_device)
    bad = order.slots.clone()
    bad[::2, 1] = order.rows.numel()
    bad[1::2, 2] = -7
    bad[3, 3] = 2 ** 31 - 1
    out, _, _ = tkq.expert_gather(x, tkq.ExpertOrder(bad, order.rows, order.offsets),
                                  out=torch.zeros(order.rows.numel(), 256, dtype=BF16, device=cuda_device))
    live = bad[(bad >= 0) & (bad < order.rows.numel())].long()
    assert float(out.float().sum()) == 256 * live.numel() and bool((out[live] == 1).all())
    y, _ = tkq.expert_reduce(out, tkq.ExpertOrder(bad, order.rows, order.offsets))
    assert torch.equal(y[:, 0].float().cpu(), ((bad >= 0) & (bad < order.rows.numel())).sum(1).float().cpu())


@pytest.mark.parametrize("T,k,E,C,align", ROWS)
@pytest.mark.parametrize("weighted,dtype", [(True, BF16), (False, BF16), (True, F32), (False, F32)])
def test_reduce(cuda_device, T, k, E, C, align, weighted, dtype):
    g = gen(C + T + 1)
    order = tkq.expert_order(ids_of(T, k, E, g).to(cuda_device), E, align)
    R = order.rows.numel()
    y = torch.randn(R, C, generator=g).bfloat16()
    y[order.rows.cpu() < 0] = float("nan")  # nothing reads the rows without a pair
    w = torch.randn(T, k, generator=g)
    slots = order.slots.cpu()
    w[slots < 0] = float("nan")
    v = torch.randn(R, generator=g)
    out, values = tkq.expert_reduce(y.to(cuda_device), order, w.to(cuda_device) if weighted else None,
                                    v.to(cuda_device), out_dtype=dtype)
    ref, size = experts64.reduce(y.nan_to_num(0.0), slots, w.nan_to_num(0.0) if weighted else None)
    close(out, ref, k * U * size + (B * ref.abs() * (1 + B) if dtype == BF16 else 0) + 1e-38)
    assert out.dtype == dtype
    assert torch.equal(values.cpu(), torch.where(slots >= 0, v[slots.clamp_min(0).long()], 0.0))
    assert torch.equal(tkq.expert_reduce(y.to(cuda_device), order, w.to(cuda_device) if weighted else None,
                                         out_dtype=dtype)[0], out)


@pytest.mark.parametrize("T,k,E,C,align", ROWS)
@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
def test_reduce_backward(cuda_device, T, k, E, C, align, fmt):
    g = gen(C + T + 2)
    order = tkq.expert_order(ids_of(T, k, E, g).to(cuda_device), E, align)
    R, end = order.rows.numel(), int(order.offsets[-1])
    slots, pair = order.slots.cpu(), order.rows.cpu()
    y, d = torch.randn(R, C, generator=g).bfloat16(), torch.randn(T, C, generator=g).bfloat16()
    y[pair < 0] = float("nan")
    w = torch.randn(T, k, generator=g)
    w[slots < 0] = float("nan")
    buf = torch.full((R, C), 0x55, dtype=torch.uint8, device=cuda_device) if fmt else \
        torch.full((R, C), GUARD, dtype=BF16, device=cuda_device)
    dy, sf, dw = tkq.expert_reduce_backward(d.to(cuda_device), y.to(cuda_device), order, w.to(cuda_device), fmt, out=buf)
    ref, ref_w, size = experts64.reduce_backward(d, y.nan_to_num(0.0), slots, w.nan_to_num(0.0))
    G = C // 128
    close(dw, ref_w, (8 * -(-G // 8) + 10) * U * size + 1e-38)
    assert bool((dw.cpu()[slots < 0] == 0).all())
    live, behind = pair >= 0, torch.arange(R) >= end
    if fmt is None:
        rows = experts64.spread(ref, slots, R)
        close(dy[:end], rows[:end], (B * (1 + B) * rows.abs() + 1e-38)[:end])
        assert bool((dy.cpu()[behind] == GUARD).all())
    else:
        prod = (w.nan_to_num(0.0).unsqueeze(2) * d.float().unsqueeze(1)).view(T * k, C).to(cuda_device)
        codes, scales = tkq.per_token_cast(prod, fmt)
        codes, scales, dy = codes.view(torch.uint8).cpu(), scales.cpu(), dy.view(torch.uint8).cpu()
        assert torch.equal(dy[live], codes[pair[live].long()])
        assert torch.equal(sf.cpu()[live], scales[pair[live].long()])
        assert not bool(dy[~live & ~behind].any()) and bool((dy[behind] == 0x55).all())


def test_gradients_against_differences(cuda_device):
    """The reduction is linear in its rows and in its weights: its differences are its gradients."""
    g = gen(5)
    T, k, E, C = 19, 3, 5, 256
    order = tkq.expert_order(ids_of(T, k, E, g).to(cuda_device), E, 16)
    R = order.rows.numel()
    y, w, d = torch.randn(R, C, generator=g).bfloat16(), torch.randn(T, k, generator=g), torch.randn(T, C, generator=g).bfloat16()
    dy, _, dw = (v if v is None else v.cpu().double() for v in tkq.expert_reduce_backward(
        d.to(cuda_device), y.to(cuda_device), order, w.to(cuda_device)))
    loss = lambda y, w: (experts64.reduce(y, order.slots.cpu(), w)[0] * d.double()).sum()
    step = torch.randn(R, C, generator=g).double()
    step[order.rows.cpu() < 0] = 0
    dy[order.rows.cpu() < 0] = 0
    diff = loss(y.double() + step, w) - loss(y, w)
    assert abs(float((dy * step).sum() - diff)) <= 2 * B * float((dy * step).abs().sum())
    step = torch.randn(T, k, generator=g).double()
    diff = loss(y, w.double() + step) - loss(y, w)
    assert abs(float((dw * step).sum() - diff)) <= 300 * U * C * float((dw * step).abs().sum() + diff.abs())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def quantized(x, fmt, dev):
    codes, sf = tkq.per_token_cast(x.bfloat16().to(dev), fmt)
    return codes, sf


def weights_of(E, N, K, g, dev, fmt="e4m3"):
    parts = [tkq.per_block_cast((torch.randn(N, K, generator=g) * (1 + e) / K ** 0.5).bfloat16().to(dev), fmt)
             for e in range(E)]
    return torch.stack([p[0].view(torch.uint8) for p in parts]).view(parts[0][0].dtype), torch.stack([p[1] for p in parts])


def starts_of(sizes, align=1):
    out = [0]
    for n in sizes:
        out.append(out[-1] + -(-n // align) * align)
    return torch.tensor(out, dtype=torch.int32)


PRODUCTS = [([1], 128, 128), ([5], 256, 256), ([128], 384, 128), ([130, 0, 5, 257], 256, 384), ([0, 0, 3], 384, 640),
            ([0, 0], 128, 256), ([300, 77, 128, 1], 640, 1024), ([1] * 70, 128, 256), ([0] * 30 + [2] * 40 + [500], 256, 128),
            ([64, 700], 1408, 768)]


@pytest.mark.parametrize("sizes,N,K", PRODUCTS)
@pytest.mark.parametrize("fmt_a,fmt_w,align", [("e4m3", "e4m3", 1), ("e5m2", "e4m3", 128), ("e4m3", "e5m2", 16)])
def test_product(cuda_device, sizes, N, K, fmt_a, fmt_w, align):
    g = gen(N + K + len(sizes))
    E = len(sizes)
    offsets = starts_of(sizes, align)
    R = int(offsets[-1]) + 3
    a, a_sf = quantized(torch.randn(R, K, generator=g) * torch.rand(R, 1, generator=g).mul(4).exp(), fmt_a, cuda_device)
    w, w_sf = weights_of(E, N, K, g, cuda_device, fmt_w)
    out = torch.full((R, N), GUARD, dtype=BF16, device=cuda_device)
    got = tkq.expert_product(a, a_sf, w, w_sf, offsets.to(cuda_device), out=out)
    assert got is out
    ref, size = experts64.product(a.cpu().float(), a_sf.cpu(), w.cpu().float(), w_sf.cpu(), offsets)
    end = int(offsets[-1])
    bound = (4 * 33 * 2 + 3 + K // 128) * U * size + B * (1 + B) * ref.abs()
    close(got[:end], ref[:end], bound[:end])
    assert bool((got[end:] == GUARD).all())
    assert tkq.tkq_read_device_status() == 0


def test_product_of_whole_numbers_is_exact(cuda_device):
    """Small whole numbers and scales of powers of two: every sum is exact, so every place counts."""
    g = gen(3)
    sizes, N, K = [200, 0, 129, 1], 384, 512
    offsets = starts_of(sizes)
    R, E = int(offsets[-1]), len(sizes)
    a = torch.randint(-3, 4, (R, K), generator=g).float()
    w = torch.randint(-2, 3, (E, N, K), generator=g).float()
    a_sf = torch.randint(-2, 3, (R, K // 128), generator=g).float().exp2()
    w_sf = torch.randint(-2, 3, (E, N // 128, K // 128), generator=g).float().exp2()
    dev = cuda_device
    got = tkq.expert_product(a.to(torch.float8_e4m3fn).to(dev), a_sf.to(dev), w.to(torch.float8_e4m3fn).to(dev),
                             w_sf.to(dev), offsets.to(dev))
    ref, _ = experts64.product(a, a_sf, w, w_sf, offsets)
    assert torch.equal(got.cpu(), ref.to(BF16))


@pytest.mark.parametrize("offsets", [[-5, 40, 10, 2000], [0, 2 ** 31 - 1, -2 ** 31, 5], [300, 300, 300, 300], [7, 9, 9, 260]])
def test_product_offsets_are_kept_in_range(cuda_device, offsets):
    g = gen(1)
    R, N, K, E = 300, 128, 256, 3
    a, a_sf = quantized(torch.randn(R, K, generator=g), "e4m3", cuda_device)
    w, w_sf = weights_of(E, N, K, g, cuda_device)
    out = torch.full((R, N), GUARD, dtype=BF16, device=cuda_device)
    tkq.expert_product(a, a_sf, w, w_sf, torch.tensor(offsets, dtype=torch.int32, device=cuda_device), out=out)
    kept = torch.tensor(offsets).clamp(0, R).cummax(0).values
    ref, size = experts64.product(a.cpu().float(), a_sf.cpu(), w.cpu().float(), w_sf.cpu(), kept)
    lo, hi = int(kept[0]), int(kept[-1])
    close(out[lo:hi], ref[lo:hi], ((4 * 33 * 2 + 3 + K // 128) * U * size + B * (1 + B) * ref.abs())[lo:hi])
    assert bool((out[:lo] == GUARD).all()) and bool((out[hi:] == GUARD).all())


GRADS = [([1], 128, 128), ([128, 0, 300], 256, 384), ([0, 0], 128, 256), ([5, 700, 0, 129], 384, 640),
         ([0] * 20 + [3], 128, 128), ([1000], 640, 256)]


@pytest.mark.parametrize("sizes,N,K", GRADS)
@pytest.mark.parametrize("fmt,dtype", [("e4m3", F32), ("e5m2", BF16)])
def test_weight_grad(cuda_device, sizes, N, K, fmt, dtype):
    g = gen(N + K)
    E = len(sizes)
    offsets = starts_of(sizes, 128)
    R = int(offsets[-1]) + 128
    dy = torch.randn(R, N, generator=g)
    x = torch.randn(R, K, generator=g)
    for e, n in enumerate(sizes):  # padding rows are zeros
        dy[int(offsets[e]) + n:int(offsets[e + 1])] = 0
        x[int(offsets[e]) + n:int(offsets[e + 1])] = 0
    dy_t, dy_sf = tkq.per_channel_cast(dy.bfloat16().to(cuda_device), fmt, transpose=True)
    x_t, x_sf = tkq.per_channel_cast(x.bfloat16().to(cuda_device), "e4m3", transpose=True)
    got = tkq.expert_weight_grad(dy_t, dy_sf, x_t, x_sf, offsets.to(cuda_device), out_dtype=dtype)
    ref, size = experts64.weight_grad(dy_t.cpu().float(), dy_sf.cpu(), x_t.cpu().float(), x_sf.cpu(), offsets)
    groups = max(sizes) // 128 + 1
    bound = (4 * 33 * 2 + 3 + groups) * U * size
    close(got, ref, bound + (B * (1 + B) * ref.abs() if dtype == BF16 else 0))
    assert got.dtype == dtype and tkq.tkq_read_device_status() == 0
    again = tkq.expert_weight_grad(dy_t, dy_sf, x_t, x_sf, offsets.to(cuda_device), out_dtype=dtype)
    assert torch.equal(got, again)


def test_weight_grad_without_rows(cuda_device):
    e = lambda *s: torch.empty(*s, dtype=torch.float8_e4m3fn, device=cuda_device)
    f = lambda *s: torch.empty(*s, device=cuda_device)
    got = tkq.expert_weight_grad(e(128, 0), f(128, 0), e(256, 0), f(256, 0),
                                 torch.zeros(4, dtype=torch.int32, device=cuda_device),
                                 out=torch.full((3, 128, 256), GUARD, device=cuda_device))
    assert not bool(got.any())


def test_data_gradient_is_the_product_with_the_transposed_matrices(cuda_device):
    g = gen(9)
    sizes, N, K = [60, 0, 200], 256, 384
    offsets = starts_of(sizes, 16)
    R, E = int(offsets[-1]), len(sizes)
    m = [torch.randn(N, K, generator=g).bfloat16() for _ in range(E)]
    w, w_sf = zip(*(tkq.per_block_cast(v.to(cuda_device)) for v in m))
    wt, wt_sf = zip(*(tkq.per_block_cast(v.t().contiguous().to(cuda_device)) for v in m))
    stack = lambda v: torch.stack([x.view(torch.uint8) for x in v]).view(torch.float8_e4m3fn)
    # the cast of the transposed matrix is the transposed cast
    assert all(torch.equal(a.view(torch.uint8).t(), b.view(torch.uint8)) and torch.equal(s.t(), t)
               for a, b, s, t in zip(w, wt, w_sf, wt_sf))
    dy, dy_sf = quantized(torch.randn(R, N, generator=g), "e5m2", cuda_device)
    got = tkq.expert_product(dy, dy_sf, stack(wt), torch.stack(wt_sf), offsets.to(cuda_device))
    ref, size = experts64.product(dy.cpu().float(), dy_sf.cpu(), stack(wt).cpu().float(), torch.stack(wt_sf).cpu(), offsets)
    close(got, ref, (4 * 33 * 2 + 3 + N // 128) * U * size + B * (1 + B) * ref.abs())
