"""The 8-bit product with a low-rank adapter a row, against 64 bits.

E is the unit roundoff of fp32.  The product and the bias carry 4 E of their
size (int -> fp32, two products, one sum).  u sums exact products (a code of 7
bits by a weight of 11) in fp32, at most K / 8 + 32 deep by any split; two more
roundings.  Its terms leave out 2^-22 of a row's largest of 32 (two of fp16,
three of bf16) or 2^-17 of each (two of bf16: two roundings of 2^-9, for 16-bit
outputs).  The sum over the ranks adds rank + 16 roundings of its size."""
import math

import pytest
import torch

from dac_vocoder_decoding_amd import vocoder as V
from test_gpu_ops import BF16, E, F16, F32, SUB, U, gelu64, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    h = V.open_ops(0)
    yield h
    torch.cuda.synchronize()
    V.voc_ops_destroy(h)


def case(g, M, N, K, rank, count, held, pad=0, offset=0):
    def codes(rows):
        x = torch.randint(-127, 128, (rows * (K + pad) + offset,), generator=g, device="cuda", dtype=torch.int8)
        return x[offset:].view(rows, K + pad)[:, :K]

    a, b = codes(M), codes(N)
    sa = torch.rand(M, generator=g, device="cuda") * 0.02 + 1e-3
    sb = torch.rand(N, generator=g, device="cuda") * 0.02 / math.sqrt(K)
    down = randn(g, count, rank, K, dtype=held, std=K ** -0.5)
    up = randn(g, count, N, rank, dtype=held, std=rank ** -0.5)
    return a, sa, b, sb, V.Adapters(down, up, torch.rand(count, generator=g, device="cuda") + 0.5), down, up


def numbers(g, M, count, pattern):
    if pattern == "runs":
        ids = (torch.arange(M, device="cuda") // 25) % (count + 1) - 1
    elif pattern == "one":
        ids = torch.full((M,), count - 1, device="cuda")
    elif pattern == "none":
        ids = torch.full((M,), -1, device="cuda")
    else:                                          # any, some of them none (too large, negative)
        ids = torch.randint(-1, count + 1, (M,), generator=g, device="cuda")
        ids[M // 2:M // 2 + 1] = 2 ** 31 - 1
        ids[M // 3:M // 3 + 1] = -2 ** 31
    return ids.to(torch.int32)


def check(y, a, sa, b, sb, ads, down, up, ids, bias, gelu):
    M, N = y.shape
    a64, b64 = a.double(), b.double()
    prod = (a64 @ b64.t()) * sa.double()[:, None] * sb.double()
    ref, size = prod + (bias.double() if bias is not None else 0.0), prod.abs() + (bias.double().abs() if bias is not None else 0.0)
    err = 4 * E * size
    rank, K = down.shape[1], down.shape[2]
    lost = 2.0 ** -17 if down.dtype == BF16 and y.dtype != F32 else 2.0 ** -22
    for i in range(ads.count):
        rows = (ids == i).nonzero()[:, 0]
        if not len(rows):
            continue
        f = (sa[rows].double() * ads.scale[i].double())[:, None]
        u, A = a64[rows] @ down[i].double().t() * f, a64[rows].abs() @ down[i].double().abs().t() * f
        w = up[i].double()
        terms = u.abs() @ w.abs().t()
        ref[rows] += u @ w.t()
        size[rows] += terms
        err[rows] += (((K / 8 + 34) * E * A) @ w.abs().t() + lost * u.abs().amax(1, keepdim=True) * w.abs().sum(1)
                      + (rank + 16) * E * terms + 2 * E * (size[rows] + terms))
    if gelu:
        err, ref = 1.13 * err + 8 * E * size, gelu64(ref)
    tol = err * (1 + U[y.dtype]) + U[y.dtype] * ref.abs() + SUB[y.dtype]
    bad = (y.double() - ref).abs() > tol
    assert not bad.any(), ((y.double() - ref).abs() / tol).max()


FORMS = [
    # M, N, K, pad, offset, the product's kernel, its shape
    (1, 1, 1, 0, 0, "product_few_shifted", (16, 16)), (3, 500, 200, 0, 0, "product_few", (16, 16)),
    (32, 4096, 1024, 0, 0, "product_few", (16, 32)), (33, 3100, 128, 0, 0, "product_few", (16, 64)),
    (64, 2000, 4096, 0, 0, "product_few", (16, 32)), (5, 1000, 333, 0, 1, "product_few_shifted", (16, 16)),
    (70, 2000, 333, 2, 5, "product_few_shifted", (16, 64)), (700, 640, 2064, 0, 0, "product_tile", (64, 64)),
    (2000, 1600, 208, 0, 16, "product_tile", (128, 64)), (2500, 2500, 400, 16, 0, "product_tile", (128, 128)),
    (3331, 3900, 272, 0, 0, "product_tile", (256, 256)), (1300, 1210, 77, 0, 0, "product_tile_rows", (64, 64)),
    (100, 20, 5000, 0, 0, "product_few", (16, 16)), (689, 1000, 1501, 6, 0, "product_tile_rows", (64, 64))]


@pytest.mark.parametrize("dtype,held", [(F32, F16), (F32, BF16), (F16, F16), (BF16, BF16), (F16, BF16)])
@pytest.mark.parametrize("M,N,K,pad,offset,kernel,shape", FORMS)
def test_matmul_int_adapters(ops, dtype, held, M, N, K, pad, offset, kernel, shape):
    """Every kernel of the product, ranks of any size, adapters in runs, one
    for all, none, and mixed from row to row."""
    g = gen(M + N + K)
    bias = randn(g, N)
    for rank, count, pattern, use, gelu in ((16, 8, "runs", bias, True), (5, 3, "any", None, False), (64, 2, "one", bias, False),
                                            (1, 1, "any", None, True), (48, 2, "none", bias, True), (100, 5, "runs", None, False)):
        if M * N > 6000000 and rank in (1, 48):
            continue
        a, sa, b, sb, ads, down, up = case(g, M, N, K, rank, count, held, pad, offset)
        ids = numbers(g, M, count, pattern)
        big = torch.full((M + 1, N + 3), 7.0, dtype=dtype, device="cuda")
        y = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, bias=use, gelu=gelu, out=big[:M, :N])
        assert V.voc_dbg_last_kernel(ops) == (kernel, shape)
        check(y, a, sa, b, sb, ads, down, up, ids, use, gelu)
        assert (big[M:] == 7).all() and (big[:, N:] == 7).all()
        none = (ids < 0) | (ids >= count)
        plain = V.matmul_int(ops, a, sa, b, sb, bias=use, gelu=gelu, dtype=dtype)
        assert torch.equal(y[none], plain[none])   # rows without an adapter: the product's own bits
        assert torch.equal(y, V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, bias=use, gelu=gelu, dtype=dtype))


@pytest.mark.parametrize("dtype,held", [(F32, F16), (BF16, BF16)])
@pytest.mark.parametrize("M,N,K,rank", [(4, 70, 300, 256), (300, 1100, 640, 256), (300, 1100, 640, 250), (600, 700, 77, 129)])
def test_adapters_of_large_rank(ops, dtype, held, M, N, K, rank):
    g = gen(rank + M)
    a, sa, b, sb, ads, down, up = case(g, M, N, K, rank, 2, held)
    ids = numbers(g, M, 2, "any")
    check(V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=dtype), a, sa, b, sb, ads, down, up, ids, None, False)


def test_adapters_that_are_not_finite_stay_with_their_rows(ops):
    g = gen(12)
    for M, N, K in ((20, 100, 130), (300, 1200, 256), (2500, 2500, 400)):
        a, sa, b, sb, ads, down, up = case(g, M, N, K, 16, 3, F16)
        ids = numbers(g, M, 3, "any")
        want = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=F32)
        down[1, 3, 5], up[2, 7, 2] = float("nan"), float("inf")
        for i in (1, 2):
            ads.set(i, down[i], up[i], ads.scale[i].item())
        y = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=F32)
        assert y[ids == 1].isnan().all()
        assert not y[ids == 2][:, 7].isfinite().any()
        kept = torch.ones(N, dtype=torch.bool, device="cuda")
        kept[7] = False
        assert torch.equal(y[ids == 2][:, kept], want[ids == 2][:, kept])
        left = (ids != 1) & (ids != 2)
        assert torch.equal(y[left], want[left])


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_adapters_of_any_size(ops, size):
    """u far outside fp16's range: scaled rows keep their terms."""
    g = gen(13)
    for M, N, K in ((20, 100, 128), (300, 1200, 256)):
        a, sa, b, sb, ads, down, up = case(g, M, N, K, 32, 2, F16)
        ads.scale.mul_(size)
        ids = numbers(g, M, 2, "one")
        y = V.matmul_int_adapters(ops, a, sa, b, sb * 0, ads, ids, dtype=F32)
        check(y, a, sa, b, sb * 0, ads, down, up, ids, None, False)


def test_adapters_of_more_rows_than_the_workspace_holds(ops):
    """Ranks of 256 in 128 MiB: 131072 rows at a time."""
    g = gen(14)
    M, N, K = 140001, 40, 48
    a, sa, b, sb, ads, down, up = case(g, M, N, K, 250, 3, BF16)
    ids, bias = numbers(g, M, 3, "runs"), randn(g, N)
    y = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, bias=bias, dtype=F16)
    check(y, a, sa, b, sb, ads, down, up, ids, bias, False)
    assert V.matmul_int_adapters(ops, a[:0], sa[:0], b, sb, ads, ids[:0]).shape == (0, N)


def test_adapters_replaced(ops):
    g = gen(15)
    a, sa, b, sb, ads, down, up = case(g, 30, 70, 100, 20, 3, BF16)
    ids = numbers(g, 30, 3, "any")
    new_down, new_up = randn(g, 7, 100, dtype=BF16), randn(g, 70, 7, dtype=BF16)
    ads.set(1, new_down, new_up, 0.25)
    down[1], up[1] = 0, 0
    down[1, :7], up[1, :, :7] = new_down, new_up
    assert ads.scale[1] == 0.25
    check(V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=F32), a, sa, b, sb, ads, down, up, ids, None, False)


def test_adapters_captured_and_replayed(ops):
    """Both launches in a graph, replayed on new rows, adapters and numbers."""
    g = gen(16)
    for M, N, K in ((8, 300, 256), (400, 700, 256)):
        a, sa, b, sb, ads, down, up = case(g, M, N, K, 16, 4, F16)
        a = a.clone()
        ids = numbers(g, M, 4, "any")
        run = lambda: V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, gelu=True)         # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        for t in range(12):
            a.copy_(torch.randint(-127, 128, a.shape, generator=g, device="cuda", dtype=torch.int8))
            ids.copy_(numbers(g, M, 4, "any"))
            ads.set(t % 4, randn(g, 16, K, dtype=F16), randn(g, N, 16, dtype=F16), 0.1 * t)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, run()), t


def test_adapters_refusals(ops):
    import ctypes
    L = V.lib()
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(64, device="cuda")
    x, ids = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 16, 64, dtype=F16, device="cuda")
    good = V.Adapters(w, torch.zeros(2, 4, 16, dtype=F16, device="cuda"))

    def mm(M=4, N=4, K=64, dtype=0, act=0, a=q.data_ptr(), adapter=ids.data_ptr(), y=x.data_ptr(), ref=None, **fields):
        c = V.voc_adapters()
        ctypes.pointer(c)[0] = good.c
        for name, value in fields.items():
            setattr(c, name, value)
        return L.vocoder_matmul_int_adapters(ops, dtype, M, N, K, a, 64, s.data_ptr(), q.data_ptr(), 64, s.data_ptr(), None, act,
                                             ctypes.byref(c) if ref is None else None, adapter, y, 64, None)

    held = dict(dtype=V.VOC_F32)
    for kw in (dict(M=-1), dict(K=0), dict(act=2), dict(a=None), dict(adapter=None), dict(adapter=ids.data_ptr() + 2), dict(y=None),
               dict(ref=0), dict(count=0), dict(count=-1), dict(rank=0), dict(rank=8), dict(rank=24), dict(rank=48), dict(rank=96), dict(rank=320),
               dict(down=None), dict(up=None), dict(down=w.data_ptr() + 8),
               dict(up=w.data_ptr() + 2), dict(scale=s.data_ptr() + 1), dict(M=1 << 24, N=1 << 24)):
        assert mm(**kw) == V.VOC_INVALID_PARAMS, kw
        assert V.voc_ops_last_error(ops), kw
    c = V.voc_adapters()
    ctypes.pointer(c)[0] = good.c
    c.dtype = held["dtype"]
    assert L.vocoder_matmul_int_adapters(ops, 0, 4, 4, 64, q.data_ptr(), 64, s.data_ptr(), q.data_ptr(), 64, s.data_ptr(), None, 0,
                                         ctypes.byref(c), ids.data_ptr(), x.data_ptr(), 64, None) == V.VOC_INVALID_PARAMS
    assert mm(M=0, a=None) == V.VOC_OK and mm() == V.VOC_OK and mm(scale=None) == V.VOC_OK


@pytest.mark.parametrize("dtype,held", [(F16, F16), (BF16, BF16), (BF16, F16)])
@pytest.mark.parametrize("rank", [3, 16, 32, 50, 64])
@pytest.mark.parametrize("pattern", ["runs of 250", "runs of 300, some none", "two mixed", "first tile only", "none"])
def test_adapters_in_tiles_of_two(ops, dtype, held, rank, pattern):
    """Tiles of 256 rows with up to two adapters, whose operands are kept in
    LDS, and tiles with more of them in the same call; ragged edges."""
    g = gen(rank)
    M, N, K, count = 3331, 3900, 272, 5
    a, sa, b, sb, ads, down, up = case(g, M, N, K, rank, count, held)
    m = torch.arange(M, device="cuda")
    if pattern == "runs of 250":
        ids = (m // 250) % count
    elif pattern == "runs of 300, some none":
        ids = (m // 300) % (count + 1) - 1
    elif pattern == "two mixed":
        ids = torch.where(torch.rand(M, generator=g, device="cuda") < 0.4, 3, torch.where(m % 7 == 0, -1, 1))
    elif pattern == "first tile only":
        ids = torch.where(m < 256, m % count, torch.where(m == 3330, 2, -1))
    else:
        ids = torch.full_like(m, -7)
    ids, bias = ids.to(torch.int32), randn(g, N)
    for width in (N, N + 3):
        big = torch.full((M + 1, width), 7.0, dtype=dtype, device="cuda")
        y = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, bias=bias, gelu=rank == 16, out=big[:M, :N])
        assert V.voc_dbg_last_kernel(ops) == ("product_tile", (256, 256))
        check(y, a, sa, b, sb, ads, down, up, ids, bias, rank == 16)
        assert (big[M:] == 7).all() and (big[:, N:] == 7).all()
        none = ids < 0
        plain = V.matmul_int(ops, a, sa, b, sb, bias=bias, gelu=rank == 16, dtype=dtype)
        assert torch.equal(y[none], plain[none])


def test_adapters_that_are_not_finite_in_tiles_of_two(ops):
    g = gen(17)
    a, sa, b, sb, ads, down, up = case(g, 3331, 3900, 272, 32, 3, BF16)
    ids = torch.where(torch.rand(3331, generator=g, device="cuda") < 0.5, 1, 2).to(torch.int32)
    ids[::5] = -1
    want = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=BF16)
    down[1, 3, 5], up[1, 7, 2] = float("nan"), float("inf")
    ads.set(1, down[1], up[1], ads.scale[1].item())
    y = V.matmul_int_adapters(ops, a, sa, b, sb, ads, ids, dtype=BF16)
    assert y[ids == 1].isnan().all() and torch.equal(y[ids != 1], want[ids != 1])
