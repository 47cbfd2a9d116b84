"""The 8-bit transformer operators against plain 64-bit implementations.

Tolerances follow from the arithmetic each operator states (fp32 sums, one
rounding of each output, fp16 probabilities): u is the unit roundoff of a
type (half a unit in the last place, relative).  Every bound is written
where it is used.
"""
import ctypes
import math

import pytest
import torch

from dac_vocoder_decoding_amd import vocoder as V

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
SUB = {F32: 0.0, F16: 2.0 ** -25, BF16: 0.0}     # half the smallest subnormal, where it matters
E = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    h = V.open_ops(0)
    yield h
    torch.cuda.synchronize()
    V.voc_ops_destroy(h)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------ rows
def check_rows(q, scale, y, rel):
    """q, scale against the exact values y [rows, C] in 64 bits, each known to
    a relative error rel of the row's largest value: the scale to rel and two
    roundings; the codes' values to half a step, 127 rel and the rounding of
    v * (1 / s)."""
    amax = y.abs().amax(1)
    s = scale.double()
    assert ((s - amax / 127).abs() <= (rel + 3 * E) * amax / 127 + 1e-300).all()
    step = 0.5 + 127 * (2 * rel + 6 * E)
    assert ((q.double() * s[:, None] - y).abs() <= step * s[:, None] + 1e-300).all()
    live = amax >= 2.0 ** -99
    assert (q[live].abs().amax(1) == 127).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,C,pad,residual", [
    (1, 1, 0, True), (3, 7, 0, False), (5, 64, 0, True), (33, 1024, 0, True), (2, 1023, 1, True),
    (7, 1501, 3, False), (4, 4096, 8, True), (3, 8192, 0, True), (2, 16384, 0, True), (2, 16383, 0, False),
    (300, 520, 0, True), (1, 2056, 0, True)])
def test_rms_norm(ops, dtype, rows, C, pad, residual):
    g = gen(rows * 131 + C)
    x = randn(g, rows, C + pad, dtype=dtype, std=3.0)[:, :C]
    r = randn(g, rows, C + pad, dtype=dtype)[:, :C] if residual else None
    w = 1 + randn(g, C, std=0.3)
    q, s, h = V.rms_norm(ops, x, w, eps=1e-5, residual=r)
    want = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(h, want)                   # one rounding of an fp32 sum
    hd = want.double()
    y = hd / (hd.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    # The fp32 sum of C squares by threads and trees: C/64 + 16 additions deep
    # at the most, halved by the square root, and six more roundings.
    check_rows(q, s, y, (C / 128 + 16) * E)


@pytest.mark.parametrize("alias", ["x", "residual"])
def test_rms_norm_in_place_and_strided(ops, alias):
    g = gen(5)
    big = randn(g, 9, 2 * 640, dtype=F16)
    x, r = big[:, :640], randn(g, 9, 640, dtype=F16)
    want = (x.float() + r.float()).half()
    w = torch.ones(640, device="cuda")
    ref = V.rms_norm(ops, x.clone(), w, residual=r.clone())
    right = big[:, 640:].clone()
    out = torch.full((9, 700), 99, dtype=torch.int8, device="cuda")
    q, s, h = V.rms_norm(ops, x, w, residual=r, h=x if alias == "x" else r, q=out[:, 3:643])
    assert h.data_ptr() == (x if alias == "x" else r).data_ptr()
    assert torch.equal(h, want) and torch.equal(q, ref[0]) and torch.equal(s, ref[1])
    assert torch.equal(big[:, 640:], right)       # the other half of the rows is untouched
    assert (out[:, :3] == 99).all() and (out[:, 643:] == 99).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,C,pad", [(1, 1, 0), (4, 5, 0), (64, 1024, 0), (3, 1000, 0), (5, 777, 2), (2, 16384, 0)])
def test_quantize_rows(ops, dtype, rows, C, pad):
    x = randn(gen(C), rows, C + pad, dtype=dtype, std=0.05)[:, :C]
    q, s = V.quantize_rows(ops, x)
    check_rows(q, s, x.double(), 0.0)


def test_rows_zero_tiny_and_non_finite(ops):
    x = torch.zeros(6, 300, device="cuda")
    x[1] = 1e-31                                  # below 2^-100: held as zeros
    x[2, 7] = float("nan")
    x[3, 299] = float("-inf")
    x[4] = 1e38
    x[5, 5] = -2.0
    q, s = V.quantize_rows(ops, x)
    assert s[0] == 0 and s[1] == 0 and not q[:4].any()
    assert s[2].isnan() and s[3].isnan()
    assert (q[4] == 127).all() and q[5, 5] == -127 and q[5].abs().sum() == 127
    w = torch.ones(300, device="cuda")
    q, s, h = V.rms_norm(ops, x, w, eps=1e-6)
    assert s[0] == 0 and not q[0].any() and not q[2:5].any()
    assert (q[1] == 127).all()                    # 1e-31 / sqrt(1e-6) = 1e-28 is above 2^-100
    assert s[2].isnan() and s[3].isnan() and s[4].isnan()   # 300 x 1e76 is beyond fp32
    assert s[5] > 0 and h.data_ptr() == x.data_ptr()
    r = torch.full((1, 300), 60000.0, device="cuda", dtype=F16)
    q, s, h = V.rms_norm(ops, r, w, residual=r)   # the sum overflows fp16
    assert h.isinf().all() and s.isnan().all() and not q.any()


def test_rows_none(ops):
    x = torch.zeros(0, 64, device="cuda")
    q, s = V.quantize_rows(ops, x)
    assert q.shape == (0, 64) and s.shape == (0,)


# --------------------------------------------------------------- product
def gelu64(x):
    return 0.5 * x * (1 + torch.erf(x / math.sqrt(2)))


def check_product(y, a, b, sa, sb, bias, gelu):
    acc = (a.cpu().to(torch.int64) @ b.cpu().to(torch.int64).t()).double()
    prod = acc * sa.cpu().double()[:, None] * sb.cpu().double()
    ref = prod + (bias.cpu().double() if bias is not None else 0.0)
    size = prod.abs() + (bias.cpu().double().abs() if bias is not None else 0.0)
    err = 4 * E * size                            # int -> fp32, two products, one sum
    if gelu:
        # slope of GELU at most 1.13; erf in fp32 to 4 units, two more products
        err = 1.13 * err + 8 * E * size
        ref = gelu64(ref)
    got = y.cpu().double()
    tol = err * (1 + U[y.dtype]) + U[y.dtype] * ref.abs() + SUB[y.dtype]
    bad = (got - ref).abs() > tol
    assert not bad.any(), ((got - ref).abs() / tol).max()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,N,K,pad,bias,gelu", [
    (1, 1, 1, 0, False, False), (1, 17, 64, 0, True, False), (3, 5, 7, 0, True, True), (16, 64, 128, 0, False, False),
    (32, 256, 1024, 0, True, True), (33, 100, 200, 3, True, False), (17, 130, 130, 0, False, True),
    (64, 128, 4096, 0, True, False), (65, 257, 1000, 0, True, False), (129, 384, 320, 16, False, False),
    (250, 300, 1501, 6, True, True), (300, 520, 576, 0, True, False), (511, 1030, 640, 0, False, False),
    (1, 1000, 8000, 0, True, False), (513, 256, 16, 0, True, False)])
def test_matmul_int(ops, dtype, M, N, K, pad, bias, gelu):
    g = gen(M * 7 + N * 3 + K)
    a = torch.randint(-127, 128, (M, K + pad), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    b = torch.randint(-127, 128, (N, K + pad), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    sa = torch.rand(M, generator=g, device="cuda") * 0.02
    sb = torch.rand(N, generator=g, device="cuda") * 0.02 / math.sqrt(K)
    bi = randn(g, N) if bias else None
    big = torch.full((M, N + 5), 7.0, dtype=dtype, device="cuda")
    y = V.matmul_int(ops, a, sa, b, sb, bias=bi, gelu=gelu, out=big[:, :N])
    check_product(y, a, b, sa, sb, bi, gelu)
    assert (big[:, N:] == 7).all()                # nothing past a row's end
    assert torch.equal(y, V.matmul_int(ops, a, sa, b, sb, bias=bi, gelu=gelu, dtype=dtype))


@pytest.mark.parametrize("M,N,K,dtype", [
    (3331, 3900, 272, BF16), (3331, 3900, 144, F32), (2500, 2500, 400, F16), (2500, 2501, 128, F32),
    (2000, 1600, 208, BF16), (2000, 1600, 1040, F32), (700, 640, 2064, F16), (1300, 1210, 77, BF16)])
def test_matmul_int_many_tiles(ops, M, N, K, dtype):
    """Sizes that fill the chip with every size of tile, with ragged edges."""
    g = gen(M + N + K)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda") / K
    y = V.matmul_int(ops, a, sa, b, sb, dtype=dtype)
    ref = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()    # integers below 2^53
    assert ((y.double() - ref).abs() <= (U[dtype] + 4 * E) * ref.abs() + SUB[dtype]).all()


def test_matmul_int_misaligned_rows(ops):
    """Rows that start at any address, a row stride that is no multiple of 16."""
    g = gen(3)
    K = 333
    a = torch.randint(-127, 128, (40 * 350 + 20,), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (70 * 341 + 20,), generator=g, device="cuda", dtype=torch.int8)
    a, b = a[5:5 + 40 * 350].view(40, 350)[:, :K], b[3:3 + 70 * 341].view(70, 341)[:, :K]
    sa, sb = torch.rand(40, device="cuda"), torch.rand(70, device="cuda")
    check_product(V.matmul_int(ops, a, sa, b, sb, dtype=F32), a, b, sa, sb, None, False)


def test_matmul_int_extreme_codes(ops):
    """-128 everywhere at the longest reduction: the sum 131071 * 2^14 fits 32 bits."""
    K = 131071
    a = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(3, device="cuda")
    y = V.matmul_int(ops, a, one[:2], b, one, dtype=F32)
    assert (y.double() - K * 2.0 ** 14).abs().max() <= E * K * 2.0 ** 14


def test_matmul_int_scale_nan_and_empty(ops):
    a = torch.zeros(3, 64, dtype=torch.int8, device="cuda")
    b = torch.ones(4, 64, dtype=torch.int8, device="cuda")
    sa = torch.tensor([1.0, float("nan"), 1.0], device="cuda")
    y = V.matmul_int(ops, a, sa, b, torch.ones(4, device="cuda"), dtype=F16)
    assert y[1].isnan().all() and (y[0] == 0).all() and (y[2] == 0).all()
    assert V.matmul_int(ops, a[:0], sa[:0], b, torch.ones(4, device="cuda"), dtype=F16).shape == (0, 4)


# ----------------------------------------------------------------- cache
def table_for(g, pages_per, spare=0):
    """A page table [B, max(pages_per) + spare] of shuffled pages; unused entries -1."""
    B, per = len(pages_per), max(pages_per) + spare
    order = torch.randperm(sum(pages_per) + 3, generator=g, device="cuda").to(torch.int32)
    t = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages_per):
        t[b, :n] = order[at:at + n]
        at += n
    return t, int(order.numel())


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def batch_of(table, past, new, **kw):
    return V.KVBatch(table, i32(past), i32(starts_of(new)), kw.get("max_new", max(new)),
                     kw.get("max_total", max(p + n for p, n in zip(past, new))))


def values_of(cache, table, b, n, which):
    """The first n tokens [kv_heads, n, D] of sequence b in 64 bits."""
    P = cache.page_tokens
    ids = table[b, :-(-n // P)].long()
    if which == "k":
        x = cache.k[ids].double() * cache.k_scale[ids].double()[..., None, None]
    else:
        x = (cache.v[ids].double() * cache.v_scale[ids].double()[..., None, None]).transpose(2, 3)
    return x.transpose(0, 1).reshape(cache.kv_heads, -1, cache.head_dim)[:, :n]


def page_scales(cache, table, b, n, which):
    ids = table[b, :-(-n // cache.page_tokens)].long()
    s = (cache.k_scale if which == "k" else cache.v_scale)[ids].double()
    return s.repeat_interleave(cache.page_tokens, 0)[:n].t()                 # [kv_heads, n]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,past,new", [
    (16, 1, 32, [0], [1]), (16, 2, 64, [0, 5], [40, 3]), (32, 3, 96, [31, 0, 32], [1, 1, 1]),
    (64, 2, 128, [100, 3, 64], [25, 0, 200]), (128, 1, 256, [5, 300], [130, 1]), (16, 5, 160, [0, 17], [16, 15])])
def test_append_holds_the_tokens(ops, dtype, P, H, D, past, new):
    """Tokens appended in two steps (the past, then the new ones), with values
    that grow so that the shared page's scale does too."""
    g = gen(P + D)
    B = len(past)
    table, pages = table_for(g, [-(-(p + n) // P) + 1 for p, n in zip(past, new)])
    cache = V.KVCache(pages, P, H, D)
    cache.k_scale.fill_(float("nan"))             # stale scales of pages without tokens are not read
    cache.v_scale.fill_(float("nan"))
    k = [randn(g, p + n, H, D, dtype=dtype) for p, n in zip(past, new)]
    v = [randn(g, p + n, H, D, dtype=dtype, std=0.3) for p, n in zip(past, new)]
    for b in range(B):
        k[b][past[b]:] *= 1.7
        v[b][past[b]:] *= 0.6
    before = cache.k.clone(), cache.v.clone()
    if sum(past):
        V.cache_append(ops, cache, batch_of(table, [0] * B, past), torch.cat([x[:p] for x, p in zip(k, past)]),
                       torch.cat([x[:p] for x, p in zip(v, past)]))
    olds = [(values_of(cache, table, b, past[b], "k"), values_of(cache, table, b, past[b], "v")) for b in range(B)]
    both = torch.cat([torch.cat((x[p:], y[p:]), 1) for x, y, p in zip(k, v, past)])     # strided views
    V.cache_append(ops, cache, batch_of(table, past, new), both[:, :H], both[:, H:])
    for b in range(B):
        n = past[b] + new[b]
        for which, x, old in (("k", k[b], olds[b][0]), ("v", v[b], olds[b][1])):
            if not n:
                continue
            got, s = values_of(cache, table, b, n, which), page_scales(cache, table, b, n, which)
            x = x.double().transpose(0, 1)
            # New tokens: half a step.  Older ones: half a step more than they were.
            tol = s[..., None] * (0.5 + 127 * 6 * E)
            assert ((got[:, past[b]:] - x[:, past[b]:]).abs() <= tol[:, past[b]:]).all()
            assert ((got[:, :past[b]] - old).abs() <= tol[:, :past[b]]).all()
            # The page's scale: the largest magnitude among the new tokens, or the older scale.
            for t0 in range(past[b] // P * P, n, P) if new[b] else ():
                lo, hi = max(t0, past[b]), min(t0 + P, n)
                amax = x[:, lo:hi].abs().amax((1, 2)) / 127
                if lo > t0:
                    older = page_scales(cache, table, b, n, which)[:, t0]
                    assert (older >= amax * (1 - 3 * E)).all()
                else:
                    assert ((s[:, lo] - amax).abs() <= 3 * E * amax).all()
    used = torch.zeros(pages, dtype=torch.bool, device="cuda")
    for b in range(B):
        used[table[b, :-(-(past[b] + new[b]) // P)].long()] = True
    assert torch.equal(cache.k[~used], before[0][~used]) and torch.equal(cache.v[~used], before[1][~used])


def test_append_requantises_exactly(ops):
    """One token after another in a page: codes and scales follow the stated
    fp32 formulas bit for bit."""
    g = gen(9)
    P, H, D = 16, 2, 64
    table, pages = table_for(g, [1])
    cache = V.KVCache(pages, P, H, D)
    x = randn(g, P, H, D) * torch.linspace(0.2, 3, P, device="cuda")[:, None, None]
    inv127 = torch.tensor(1 / 127, dtype=F32, device="cuda")
    codes = torch.zeros(H, P, D, device="cuda")
    scale = torch.zeros(H, device="cuda")
    for t in range(P):
        V.cache_append(ops, cache, batch_of(table, [t], [1]), x[t:t + 1], x[t:t + 1])
        now = torch.maximum(scale, x[t].abs().amax(1) * inv127)
        inv = torch.ones_like(now) / now
        codes[:, :t] = (codes[:, :t] * (scale * inv)[:, None, None]).round()
        codes[:, t] = (x[t] * inv[:, None]).round().clamp(-127, 127)
        scale = now
        page = int(table[0, 0])
        assert torch.equal(cache.k_scale[page], scale) and torch.equal(cache.v_scale[page], scale)
        assert torch.equal(cache.k[page].float(), codes)
        assert torch.equal(cache.v[page].transpose(1, 2).float(), codes)


def test_append_non_finite_and_zero(ops):
    g = gen(10)
    P, H, D = 16, 3, 32
    table, pages = table_for(g, [2])
    cache = V.KVCache(pages, P, H, D)
    k = randn(g, 20, H, D, dtype=F16)
    k[:, 1] = 0
    k[2, 2, 5] = float("nan")
    k[17, 0, 1] = float("inf")
    V.cache_append(ops, cache, batch_of(table, [0], [20]), k, k)
    p0, p1 = int(table[0, 0]), int(table[0, 1])
    for s, c in ((cache.k_scale, cache.k), (cache.v_scale, cache.v)):
        assert s[p0, 0] > 0 and s[p1, 2] > 0
        assert s[p0, 1] == 0 and s[p1, 1] == 0 and not c[p0, 1].any()
        assert s[p0, 2].isnan() and s[p1, 0].isnan() and not c[p0, 2].any()
    V.cache_append(ops, cache, batch_of(table, [20], [1]), torch.ones_like(k[:1]), torch.ones_like(k[:1]))
    assert cache.k_scale[p1, 0].isnan()           # a page once NaN stays so while it holds that token
    assert cache.k_scale[p1, 1] == torch.tensor(1 / 127, dtype=F32)


def test_append_stays_inside_the_table(ops):
    """Positions past the table, pages out of range and sequences whose rows
    are out of bounds append nothing."""
    g = gen(11)
    P, H, D = 16, 1, 32
    cache = V.KVCache(4, P, H, D)
    cache.k.fill_(5)
    k = randn(g, 30, H, D)
    table = i32([[0, 7], [-1, 1], [2, 3]])
    starts = i32([0, 20, 25, 99])                 # the last sequence's rows end past the 30
    b = V.KVBatch(table, i32([20, 0, 0]), starts, 20, 40)
    V.cache_append(ops, cache, b, k, k)
    torch.cuda.synchronize()
    assert (cache.k == 5).all() and not cache.k_scale.any()
    b = V.KVBatch(table, i32([20, 0, 0]), i32([0, 20, 25, 30]), 4, 40)   # more new tokens than max_new
    V.cache_append(ops, cache, b, k, k)
    assert (cache.k == 5).all()


# ------------------------------------------------------------- attention
def attend64(cache, table, past, new, q, scale, causal, window):
    """Plain attention in 64 bits over the dequantised cache, and the bound of
    the kernel's error for each output.

    With p the probabilities and A = sum p |v| / sum p: a relative error e_p
    of every p moves an output by at most 2 e_p A.  The scores are off by
    delta = (D + 8) E scale sum |q k| (fp32 sums; for fp32 queries also the 22
    bits that two fp16 terms hold, 4 E of the same sum), so e_p = delta + the
    exponential's 2^-21 (its argument, up to 2^7 in size, in fp32) + the
    rounding of p to fp16 (2^-11) or two terms (2^-21); the sums of n terms
    add n / 64 + 32 roundings each."""
    Hq, H = q.shape[1], cache.kv_heads
    outs, tols = [], []
    base = 0
    for b in range(len(past)):
        total = past[b] + new[b]
        rows = q[base:base + new[b]].double().transpose(0, 1)                # [Hq, n, D]
        base += new[b]
        if not new[b]:
            continue
        k = values_of(cache, table, b, total, "k").repeat_interleave(Hq // H, 0)
        v = values_of(cache, table, b, total, "v").repeat_interleave(Hq // H, 0)
        at = past[b] + torch.arange(new[b], device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        seen = torch.ones(new[b], total, dtype=torch.bool, device="cuda")
        if causal:
            seen &= j <= at
        if window:
            seen &= j > at - window
        z = (rows @ k.transpose(1, 2)) * scale
        z = z.masked_fill(~seen, -math.inf)
        p = torch.softmax(z, -1)
        D = q.shape[2]
        delta = (D + 8 + 4) * E * abs(scale) * (rows.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
        two = q.dtype == F32
        e_p = delta + 2.0 ** -21 + (2.0 ** -21 if two else 2.0 ** -11) + (total / 64 + 32) * E
        o = p @ v
        A = p @ v.abs()
        outs.append(o.transpose(0, 1))
        tols.append((2 * e_p * A + U[q.dtype] * o.abs() + SUB[q.dtype]
                     + total * 2.0 ** -36 * v.abs().amax((1, 2), keepdim=True)).transpose(0, 1))
    return torch.cat(outs), torch.cat(tols)


def filled(g, P, H, D, past, new, spread=1.0):
    total = [p + n for p, n in zip(past, new)]
    table, pages = table_for(g, [max(1, -(-t // P)) for t in total], spare=1)
    cache = V.KVCache(pages, P, H, D)
    cache.k.copy_(torch.randint(-127, 128, cache.k.shape, generator=g, device="cuda", dtype=torch.int8))
    cache.v.copy_(torch.randint(-127, 128, cache.v.shape, generator=g, device="cuda", dtype=torch.int8))
    cache.k_scale.copy_(torch.exp(randn(g, pages, H, std=0.5)) * spread / 70)
    cache.v_scale.copy_(torch.exp(randn(g, pages, H, std=2.0)) / 70)
    # Pages that hold no token carry NaN scales: nothing may read them.
    idle = torch.ones(pages, dtype=torch.bool, device="cuda")
    for b, t in enumerate(total):
        idle[table[b, :-(-t // P)].long()] = False
    cache.k_scale[idle] = float("nan")
    cache.v_scale[idle] = float("nan")
    return cache, table


ATTEND = [
    # P, kv heads, D, group, past, new, causal, window
    (16, 1, 32, 1, [0], [1], True, 0),
    (16, 2, 64, 1, [1, 63, 64, 65], [1, 1, 1, 1], True, 0),
    (64, 2, 128, 4, [700, 3], [1, 1], True, 0),
    (32, 1, 96, 5, [129], [1], True, 0),
    (128, 3, 64, 2, [5, 1000, 0], [3, 7, 0], True, 0),
    (16, 2, 64, 1, [100, 40], [25, 19], True, 72),
    (32, 2, 128, 2, [0, 0], [70, 33], True, 0),
    (64, 1, 256, 3, [0], [150], True, 0),
    (16, 1, 160, 1, [17], [40], False, 0),
    (32, 1, 192, 2, [50], [33], False, 20),
    (16, 1, 224, 7, [3], [20], True, 1),
    (64, 2, 128, 1, [0, 10], [300, 257], True, 0),
    (64, 1, 128, 4, [0], [200], True, 33),
    (128, 1, 64, 16, [2000], [1], True, 0),
    (32, 1, 64, 40, [90], [2], True, 0),
    (64, 1, 64, 1, [5000], [1], True, 0),
    (64, 2, 64, 1, [130], [130], False, 0),
    # Enough rows and keys for the kernel of many rows (whole, then in parts),
    # every size of head, windows, ragged tiles and pages.
    (64, 8, 128, 2, [0, 37], [1300, 1111], True, 0),
    (32, 2, 96, 1, [1], [2500], True, 0),
    (16, 16, 64, 1, [0, 3], [2049, 1900], True, 0),
    (128, 16, 32, 1, [0], [2900], False, 0),
    (64, 2, 256, 1, [0], [2300], True, 0),
    (32, 2, 224, 1, [9], [2301], True, 0),
    (16, 2, 160, 1, [2000], [1500], True, 0),
    (64, 4, 192, 1, [100], [1500], False, 0),
    (64, 4, 128, 8, [9000], [40], True, 0),
    (16, 8, 128, 4, [5], [1700], True, 700),
    (64, 8, 64, 2, [6000, 100, 5000], [300, 0, 299], True, 0),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,group,past,new,causal,window", ATTEND)
def test_attention(ops, dtype, P, H, D, group, past, new, causal, window):
    g = gen(P * 3 + D + sum(past) + sum(new))
    cache, table = filled(g, P, H, D, past, new)
    q = randn(g, sum(new), H * group, D, dtype=dtype)
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q, causal=causal, window=window)
    ref, tol = attend64(cache, table, past, new, q, D ** -0.5, causal, window)
    worst = ((o.double() - ref).abs() / tol).max().item()
    assert worst <= 1, worst
    assert torch.equal(o, V.cache_attention(ops, cache, batch_of(table, past, new), q, causal=causal, window=window))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_attention_sharp_scores(ops, dtype):
    """Scores of hundreds: the maximum moves far and often, most probabilities vanish."""
    g = gen(77)
    cache, table = filled(g, 32, 2, 64, [400, 900], [30, 1], spread=30.0)
    q = randn(g, 31, 4, 64, dtype=dtype, std=4.0)
    o = V.cache_attention(ops, cache, batch_of(table, [400, 900], [30, 1]), q)
    ref, tol = attend64(cache, table, [400, 900], [30, 1], q, 0.125, True, 0)
    assert ((o.double() - ref).abs() <= tol).all()


def test_attention_query_ranges(ops):
    """Rows of very large, very small and zero queries, in types that hold them."""
    g = gen(78)
    cache, table = filled(g, 16, 1, 64, [60], [6])
    q = randn(g, 6, 1, 64)
    gain = torch.tensor([1e30, 1e-30, 0.0, 1.0, 1e-38, 1e4], device="cuda")[:, None, None]
    for dtype in (F32, BF16):
        x = (q * gain).to(dtype)
        o = V.cache_attention(ops, cache, batch_of(table, [60], [6]), x, scale=1e-3)
        ref, tol = attend64(cache, table, [60], [6], x, 1e-3, True, 0)
        # A score of 1e28 leaves one key; ties cannot be told from near ties there.
        assert ((o.double() - ref).abs() <= tol)[1:].all()
        assert torch.isfinite(o).all()


def test_attention_strided_and_rows_between(ops):
    """q and o as slices of wider rows; rows that belong to no sequence stay as they are."""
    g = gen(79)
    past, new = [33, 5], [4, 2]
    cache, table = filled(g, 16, 2, 64, past, new)
    big = randn(g, 9, 3, 4, 64, dtype=F16)
    q = big[:, 1]                                  # token stride 3 * 4 * 64
    out = torch.full((9, 4, 2, 64), 9.0, dtype=F16, device="cuda")[:, :, 0]
    b = V.KVBatch(table, i32(past), i32([1, 5, 7]), 4, 64)
    V.cache_attention(ops, cache, b, q, out=out)
    ref, tol = attend64(cache, table, past, new, q[1:7], 0.125, True, 0)
    assert ((out[1:7].double() - ref).abs() <= tol).all()
    assert (out[0] == 9).all() and (out[7:] == 9).all()


def test_attention_empty_rows_and_missing_pages(ops):
    """Missing pages hold no tokens; a query that sees none gives zeros."""
    g = gen(80)
    P, H, D = 16, 1, 64
    cache, table = filled(g, P, H, D, [96], [3])
    q = randn(g, 3, 2, D)
    hole = table.clone()
    hole[0, 1] = -1
    hole[0, 3] = 1 << 30
    full = V.cache_attention(ops, cache, batch_of(hole, [96], [3]), q)
    keep = [i for i in range(7) if i not in (1, 3)]
    k, v = values_of(cache, table, 0, 99, "k")[0], values_of(cache, table, 0, 99, "v")[0]
    seen = torch.zeros(3, 99, dtype=torch.bool, device="cuda")
    for i in keep:
        seen[:, i * P:(i + 1) * P] = True
    seen &= torch.arange(99, device="cuda")[None] <= 96 + torch.arange(3, device="cuda")[:, None]
    z = (torch.einsum("thd,nd->htn", q.double().cpu(), k.cpu()) / 8).masked_fill(~seen.cpu(), -math.inf)
    ref = torch.einsum("htn,nd->thd", torch.softmax(z, -1), v.cpu())
    # fp32 queries: the bound of attend64 for such sizes, 2 e_p A with e_p below 2^-15 here
    assert ((full.double().cpu() - ref).abs() <= 2.0 ** -14 * v.abs().max().cpu()).all()
    none = torch.full_like(table, -1)
    o = V.cache_attention(ops, cache, batch_of(none, [96], [3]), q, out=torch.full_like(q, 3.0))
    assert (o == 0).all()
    # A window that lies in a missing page.
    hole = table.clone()
    hole[0, 6] = -1
    o = V.cache_attention(ops, cache, batch_of(hole, [96], [3]), q, window=2)
    assert (o[1:] == 0).all() and (o[0] != 0).any()


@pytest.mark.parametrize("dtype", [F32, F16])
def test_attention_non_finite_pages(ops, dtype):
    """A page whose scale is NaN makes NaN what sees it and nothing else, also
    inside one tile of queries."""
    g = gen(81)
    past, new = [64], [64]
    cache, table = filled(g, 16, 2, 64, past, new)
    q = randn(g, 64, 4, 64, dtype=dtype)
    ref, tol = attend64(cache, table, past, new, q, 0.125, True, 0)
    for s in (cache.k_scale, cache.v_scale):
        kept = s.clone()
        s[int(table[0, 6]), 1] = float("nan")      # positions 96 .. 111, cache head 1
        o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
        bad = torch.zeros(64, 4, dtype=torch.bool, device="cuda")
        bad[32:, 2:] = True
        assert o[bad].isnan().all()
        assert ((o.double() - ref).abs() <= tol)[~bad].all()
        s.copy_(kept)
    q[5, 1, 3] = float("nan")
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
    bad = torch.zeros(64, 4, dtype=torch.bool, device="cuda")
    bad[5, 1] = True
    assert o[bad].isnan().all() and ((o.double() - ref).abs() <= tol)[~bad].all()


def test_append_then_attend_by_chunks(ops):
    """A prompt in one call and the same tokens frame by frame: the caches
    differ only by the codes' growth of scale, the outputs accordingly."""
    g = gen(82)
    H, D, P, n = 2, 64, 16, 50
    x = [randn(g, n, H, D, dtype=F16) for _ in range(3)]
    outs = []
    for step in (n, 1, 7):
        table, pages = table_for(gen(5), [-(-n // P)])
        cache = V.KVCache(pages, P, H, D)
        o = []
        for t in range(0, n, step):
            m = min(step, n - t)
            b = batch_of(table, [t], [m])
            V.cache_append(ops, cache, b, x[1][t:t + m], x[2][t:t + m])
            o.append(V.cache_attention(ops, cache, b, x[0][t:t + m]))
        outs.append(torch.cat(o).double())
    # Each growth of a page's scale rounds its older codes by half a step, at
    # most 15 times in a page of 16; a step is max|v| / 127, and a key's
    # error moves its score by at most as much times |q|_1 / sqrt(D).  The
    # whole prompt's page scale also covers tokens that a frame does not see.
    step = 4.5 / 127
    tol = 16 * 0.5 * step * (1 + 4.5 * 64 * 0.8 / 8)
    assert (outs[1] - outs[0]).abs().max() <= tol and (outs[2] - outs[0]).abs().max() <= tol
    # In the mean they are far closer: a few per cent.
    assert (outs[1] - outs[0]).norm() <= 0.1 * outs[0].norm()
    assert (outs[2] - outs[0]).norm() <= 0.1 * outs[0].norm()


def test_cache_beyond_4_gib(ops):
    """Pages whose codes lie past 32-bit byte offsets, for both attention kernels."""
    g = gen(85)
    P, H, D = 128, 8, 256
    pages = 17000                                  # 4.4 GB of key codes
    cache = V.KVCache.from_tensors(
        torch.empty(pages, H, P, D, dtype=torch.int8, device="cuda"),
        torch.empty(pages, H, D, P, dtype=torch.int8, device="cuda"),
        torch.full((pages, H), float("nan"), device="cuda"), torch.full((pages, H), float("nan"), device="cuda"))
    for n in (200, 1500):
        used = -(-n // P)
        table = torch.arange(pages - used, pages, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
        k, v, q = (randn(g, n, H, D, dtype=F16) for _ in range(3))
        b = batch_of(table, [0], [n])
        V.cache_append(ops, cache, b, k, v)
        o = V.cache_attention(ops, cache, b, q)
        ref, tol = attend64(cache, table, [0], [n], q, 1 / 16, True, 0)
        assert ((o.double() - ref).abs() <= tol).all()
        got = values_of(cache, table, 0, n, "v").transpose(0, 1)
        assert ((got - v.double()).abs() <= page_scales(cache, table, 0, n, "v").t()[..., None] * (0.5 + 127 * 6 * E)).all()


# ------------------------------------------------- streams, graphs, errors
def test_on_another_stream(ops):
    g = gen(83)
    past, new = [500, 20], [1, 1]
    cache, table = filled(g, 32, 2, 64, past, new)
    q = randn(g, 2, 8, 64, dtype=F16)
    x, w = randn(g, 2, 512, dtype=F16), torch.ones(512, device="cuda")
    want = V.cache_attention(ops, cache, batch_of(table, past, new), q)
    rows = V.rms_norm(ops, x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.empty_like(q)
    b = batch_of(table, past, new)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late.copy_(q)                              # the operator has to come after this
        got = V.cache_attention(ops, cache, b, late)
        got_rows = V.rms_norm(ops, x, w)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(got_rows[0], rows[0])
    explicit = V.cache_attention(ops, cache, b, q, stream=s)
    s.synchronize()
    assert torch.equal(explicit, want)


def test_graph_replays_equal_eager(ops):
    """One layer's worth of calls captured once and replayed on new inputs,
    with eager calls between the replays."""
    g = gen(84)
    H, D, P, B, C = 2, 64, 16, 3, 256
    table, pages = table_for(g, [40] * B)
    cache, eager_cache = V.KVCache(pages, P, H, D), V.KVCache(pages, P, H, D)
    past = torch.zeros(B, dtype=torch.int32, device="cuda")
    starts = i32([0, 1, 2, 3])
    x = randn(g, B, C, dtype=F16)
    wq, ws = V.quantize_rows(ops, randn(g, 3 * H * D, C, std=0.1))
    w = torch.ones(C, device="cuda")

    def step(cache, past):
        b = V.KVBatch(table, past, starts, 1, 40 * P)
        q, s, _ = V.rms_norm(ops, x, w)
        qkv = V.matmul_int(ops, q, s, wq, ws, dtype=F16).view(B, 3 * H, D)
        V.cache_append(ops, cache, b, qkv[:, H:2 * H], qkv[:, 2 * H:])
        return V.cache_attention(ops, cache, b, qkv[:, :H]), b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, keep0 = step(V.KVCache(pages, P, H, D), past)     # warm up on another cache
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, keep = step(cache, past)
    for t in range(20):
        x.copy_(randn(g, B, C, dtype=F16))
        past.fill_(t * 31)
        graph.replay()
        want, _ = step(eager_cache, past)
        torch.cuda.synchronize()
        assert torch.equal(out, want), t
        assert torch.equal(cache.k, eager_cache.k) and torch.equal(cache.v_scale, eager_cache.v_scale), t


def test_handles_and_refusals(ops):
    L = V.lib()
    st, h = V.voc_ops_create(-1)
    assert st == V.VOC_INVALID_PARAMS and not h.value and "device" in V.voc_ops_last_error(None)
    assert V.voc_ops_create(4096)[0] == V.VOC_INVALID_PARAMS
    x = torch.zeros(4, 64, device="cuda")
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(64, device="cuda")

    def norm(dtype=0, rows=4, C=64, xp=x.data_ptr(), ldx=64, r=None, ldr=0, hp=None, ldh=0, w=s.data_ptr(), eps=1e-6,
             qp=q.data_ptr(), ldq=64, sp=s.data_ptr()):
        return L.vocoder_rms_norm(ops, dtype, rows, C, xp, ldx, r, ldr, hp, ldh, w, eps, qp, ldq, sp, None)

    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(C=0), dict(C=16385), dict(xp=None), dict(ldx=63),
               dict(r=x.data_ptr(), ldr=1), dict(hp=x.data_ptr(), ldh=2), dict(w=None), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(qp=None), dict(ldq=63), dict(sp=None),
               dict(xp=x.data_ptr() + 1), dict(sp=s.data_ptr() + 2), dict(ldx=1 << 41)):
        assert norm(**kw) == V.VOC_INVALID_PARAMS, kw
        assert V.voc_ops_last_error(ops), kw
    assert norm(rows=0, xp=None) == V.VOC_OK
    assert V.voc_ops_last_error(ops) == ""

    def mm(dtype=0, M=4, N=4, K=64, a=q.data_ptr(), lda=64, sa=s.data_ptr(), b=q.data_ptr(), ldb=64, sb=s.data_ptr(),
           bias=None, act=0, y=x.data_ptr(), ldy=64):
        return L.vocoder_matmul_int(ops, dtype, M, N, K, a, lda, sa, b, ldb, sb, bias, act, y, ldy, None)

    for kw in (dict(dtype=7), dict(M=-1), dict(N=-1), dict(K=0), dict(K=131072), dict(a=None), dict(lda=63),
               dict(sa=None), dict(b=None), dict(ldb=1), dict(sb=None), dict(act=2), dict(y=None), dict(ldy=3),
               dict(bias=s.data_ptr() + 1), dict(y=x.data_ptr() + 2)):
        assert mm(**kw) == V.VOC_INVALID_PARAMS, kw

    cache = V.KVCache(4, 16, 2, 64)
    table, one, st3 = i32([[0, 1]]), i32([0]), i32([0, 1])
    kv = torch.zeros(1, 2, 64, device="cuda")

    def with_cache(call, **kw):
        c, b = V.voc_kv_cache(), V.voc_kv_batch()
        ctypes.pointer(c)[0] = cache.c
        ctypes.pointer(b)[0] = V.KVBatch(table, one, st3, 1, 1).c
        b.tokens = 1
        for k, v in kw.items():
            setattr(c if hasattr(c, k) else b, k, v)
        if call == "append":
            return L.vocoder_cache_append(ops, ctypes.byref(c), ctypes.byref(b), 0, kv.data_ptr(), 128, 64, kv.data_ptr(),
                                          128, 64, None)
        return L.vocoder_cache_attention(ops, ctypes.byref(c), ctypes.byref(b), 0, 2, kv.data_ptr(), 128, 64, 1.0, 1, 0,
                                         kv.data_ptr(), 128, 64, None)

    for kw in (dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256), dict(head_dim=48), dict(head_dim=288),
               dict(head_dim=0), dict(kv_heads=0), dict(n_pages=0), dict(k=None), dict(v=None), dict(k_scale=None),
               dict(v_scale=None), dict(k=cache.k.data_ptr() + 8), dict(batch=-1), dict(batch=70000), dict(tokens=-1),
               dict(max_new=-1), dict(max_total=-1), dict(table_stride=0), dict(table_stride=1 << 30),
               dict(starts=None), dict(past=None), dict(page_table=None), dict(past=one.data_ptr() + 2)):
        for call in ("append", "attend"):
            assert with_cache(call, **kw) == V.VOC_INVALID_PARAMS, (call, kw)
            assert V.voc_ops_last_error(ops)
    for call in ("append", "attend"):
        assert with_cache(call, batch=0) == V.VOC_OK and with_cache(call, tokens=0) == V.VOC_OK

    b = V.KVBatch(table, one, st3, 1, 1)
    b.c.tokens = 1

    def attend(dtype=0, heads=2, qp=kv.data_ptr(), qt=128, qhs=64, scale=1.0, causal=1, window=0, o=kv.data_ptr(),
               ot=128, oh=64):
        return L.vocoder_cache_attention(ops, cache.ref, b.ref, dtype, heads, qp, qt, qhs, scale, causal, window, o, ot,
                                         oh, None)

    for kw in (dict(dtype=5), dict(heads=0), dict(heads=3), dict(heads=1), dict(qp=None), dict(qp=kv.data_ptr() + 4),
               dict(qt=127), dict(qhs=-64), dict(scale=float("inf")), dict(causal=2), dict(window=-1), dict(o=None),
               dict(ot=66), dict(oh=1)):
        assert attend(**kw) == V.VOC_INVALID_PARAMS, kw
    assert L.vocoder_cache_append(ops, None, b.ref, 0, kv.data_ptr(), 1, 1, kv.data_ptr(), 1, 1, None) == \
        V.VOC_INVALID_PARAMS
    assert L.vocoder_cache_append(ops, cache.ref, b.ref, 0, kv.data_ptr() + 2, 1, 1, kv.data_ptr(), 1, 1, None) == \
        V.VOC_INVALID_PARAMS


def test_binding_refuses_what_the_library_cannot_see(ops):
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        V.rms_norm(ops, x, w[:63])
    with pytest.raises(ValueError):
        V.rms_norm(ops, x, w, residual=x[:3])
    with pytest.raises(ValueError):
        V.rms_norm(ops, x.t(), w)
    with pytest.raises(ValueError):
        V.rms_norm(ops, x.double(), w)
    with pytest.raises(ValueError):
        V.quantize_rows(ops, x, q=torch.zeros(4, 63, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError):
        V.quantize_rows(ops, x.cpu())
    q, s = V.quantize_rows(ops, x)
    with pytest.raises(ValueError):
        V.matmul_int(ops, q, s, q[:, :32], s)
    with pytest.raises(ValueError):
        V.matmul_int(ops, q, s[:3], q, s)
    with pytest.raises(ValueError):
        V.matmul_int(ops, q, s, q, s, out=torch.zeros(4, 5, device="cuda"))
    cache = V.KVCache(2, 16, 2, 64)
    b = V.KVBatch(i32([[0]]), i32([0]), i32([0, 1]), 1, 1)
    with pytest.raises(ValueError):
        V.cache_append(ops, cache, b, torch.zeros(1, 2, 32, device="cuda"), torch.zeros(1, 2, 32, device="cuda"))
    with pytest.raises(ValueError):
        V.cache_attention(ops, cache, b, torch.zeros(1, 2, 32, device="cuda"))
    with pytest.raises(ValueError):
        V.KVBatch(i32([[0]]).long(), i32([0]), i32([0, 1]), 1, 1)
    with pytest.raises(ValueError):
        V.KVBatch(i32([[0]]), i32([0]), i32([0]), 1, 1)
    with pytest.raises(ValueError):
        V.KVCache.from_tensors(cache.k, cache.k, cache.k_scale, cache.v_scale)


def test_calls_too_large_for_one_launch_are_refused(ops):
    L = V.lib()
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(64, device="cuda")
    for M, N in ((1 << 24, 1 << 24), ((1 << 12) * 64, (1 << 11) * 64)):
        assert L.vocoder_matmul_int(ops, 0, M, N, 64, q.data_ptr(), 64, s.data_ptr(), q.data_ptr(), 64, s.data_ptr(), None,
                                    0, s.data_ptr(), N, None) == V.VOC_INVALID_PARAMS, (M, N)
        assert "too many" in V.voc_ops_last_error(ops)
    cache = V.KVCache(2, 16, 2, 64)
    kv = torch.zeros(1, 2, 64, device="cuda")
    for batch, max_new in ((65535, 2048), (1, 1 << 24)):
        b = V.KVBatch(i32([[0]]), i32([0]), i32([0, 1]), max_new, 1)
        b.c.tokens, b.c.batch = 1, batch
        heads = 2 if batch > 1 else 64
        assert L.vocoder_cache_attention(ops, cache.ref, b.ref, 0, heads, kv.data_ptr(), 128, 64, 1.0, 1, 0, kv.data_ptr(),
                                         128, 64, None) == V.VOC_INVALID_PARAMS, (batch, max_new)
        assert "too many" in V.voc_ops_last_error(ops)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,group,past,new,causal,window", [
    (64, 1, 64, 16, [40000], [1], True, 0), (32, 1, 32, 1, [20000], [1], True, 0), (128, 1, 96, 3, [9000, 20], [1, 1], True, 0),
    (64, 1, 160, 2, [9000], [3], False, 0), (16, 1, 256, 2, [3000], [9], True, 1500), (16, 2, 64, 1, [400, 700], [40, 1], True, 0),
    (32, 1, 224, 5, [600], [7], True, 0), (64, 2, 192, 2, [10, 8000], [1, 1], True, 0)])
def test_attention_joins(ops, dtype, P, H, D, group, past, new, causal, window):
    """Caches whose keys are split: one row and sixteen to a tile, few parts and many, sequences with empty parts."""
    test_attention(ops, dtype, P, H, D, group, past, new, causal, window)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,C,pad,residual", [(5, 1025, 0, True), (9, 2048, 0, True), (3, 2047, 1, False), (2500, 1504, 8, True)])
def test_rms_norm_of_four_waves(ops, dtype, rows, C, pad, residual):
    test_rms_norm(ops, dtype, rows, C, pad, residual)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("past,new", [([0, 60], [12, 5]), ([0, 60], [13, 6]), ([64, 127], [8, 12])])
def test_append_of_a_few_tokens(ops, dtype, past, new):
    test_append_holds_the_tokens(ops, dtype, 64, 2, 96, past, new)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,D,past,new,causal,window", [
    (16, 64, 0, 250, True, 0), (32, 256, 0, 90, True, 0), (64, 64, 3, 140, True, 72), (128, 96, 30, 100, False, 0)])
def test_attention_many_short_prompts(ops, dtype, P, D, past, new, causal, window):
    """A tile of rows to each of 16 heads of 16 sequences of different lengths, some without new tokens."""
    test_attention(ops, dtype, P, 16, D, 1, [past * i for i in range(16)], [0 if i % 7 == 3 else new - 5 * i for i in range(16)],
                   causal, window)


def attend64_by_keys(cache, table, past, new, q, scale, causal, window, two=None, hole=()):
    """Plain attention in 64 bits, with the bound of attend64 taken key by key
    (an error e of a probability p moves the output by at most p e (|v| + |o|))
    and fp16's last step as the kernels state it: 2^-35 of the row's largest
    p times value scale for each key, times its code.  `hole`: (sequence, column)
    of pages that are missing from the table that the kernel was given."""
    Hq, H, D = q.shape[1], cache.kv_heads, q.shape[2]
    outs, tols, base = [], [], 0
    for b in range(len(past)):
        total = past[b] + new[b]
        rows = q[base:base + new[b]].double().transpose(0, 1)                # [Hq, n, D]
        base += new[b]
        if not new[b]:
            continue
        k = values_of(cache, table, b, total, "k").repeat_interleave(Hq // H, 0).transpose(1, 2).contiguous()
        v = values_of(cache, table, b, total, "v").repeat_interleave(Hq // H, 0)
        vs = page_scales(cache, table, b, total, "v").repeat_interleave(Hq // H, 0)[:, None]
        at = past[b] + torch.arange(new[b], device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        seen = torch.ones(new[b], total, dtype=torch.bool, device="cuda")
        if causal:
            seen &= j <= at
        if window:
            seen &= j > at - window
        for c in (c for s, c in hole if s == b):
            seen[:, c * cache.page_tokens:(c + 1) * cache.page_tokens] = False
        p = torch.softmax(((rows @ k) * scale).masked_fill(~seen, -math.inf), -1)
        p = torch.where(seen.any(-1, keepdim=True), p, 0.0)
        two = q.dtype == F32 if two is None else two
        e = (D + 8 + 4) * E * abs(scale) * (rows.abs() @ k.abs()) + 2.0 ** -21 + (2.0 ** -21 if two else 2.0 ** -11) \
            + (total / 64 + 32) * E
        o = p @ v
        outs.append(o.transpose(0, 1))
        tols.append(((p * e) @ v.abs() + (p * e).sum(-1, keepdim=True) * o.abs() + U[q.dtype] * o.abs() + SUB[q.dtype]
                     + total * 2.0 ** -35 * 127 * (p * vs).amax(-1, keepdim=True)).transpose(0, 1))
    return torch.cat(outs), torch.cat(tols)


@pytest.mark.parametrize("dtype,ratio,push", [(F32, 20, 1.2), (F32, 40, 2.0), (F32, 70, 3.6), (F16, 20, 1.2),
                                              (BF16, 20, 1.2), (BF16, 70, 3.6)])
@pytest.mark.parametrize("P,H,D,past,new", [
    (16, 2, 64, [200, 90], [1, 5]),                             # few rows
    (16, 16, 64, [3 * i for i in range(16)], [250] * 16),       # many rows
    (32, 16, 128, [0] * 17, [130] * 17)])
def test_attention_value_scales_far_apart(ops, dtype, P, H, D, past, new, ratio, push):
    """Pages whose value scales are 2^20, 2^40 and 2^70 times the others' and
    whose keys the queries point away from (probabilities of about 2^-25,
    2^-42 and 2^-75): they count for what they weigh, and no more."""
    g = gen(91 + ratio)
    cache, table = filled(g, P, H, D, past, new)
    cache.v_scale.copy_(torch.rand(cache.v_scale.shape, generator=g, device="cuda") * 0.01 + 0.01)
    cache.k_scale.fill_(1 / 70)
    far = torch.stack([table[:, 0], table[:, 3]], 1).long()
    cache.k[far] = -127
    cache.v_scale[far] *= 2.0 ** ratio
    if dtype == F16:
        cache.v_scale.mul_(2.0 ** -6)               # 0.02 * 2^20 * 127 fits fp16 then
    q = (randn(g, sum(new), H, D, std=0.3) + push * (64 / D) ** 0.5).to(dtype)
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
    ref, tol = attend64_by_keys(cache, table, past, new, q, D ** -0.5, True, 0)
    worst = ((o.double() - ref).abs() / tol).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("P,H,D,past,new,causal", [
    (16, 2, 64, [300], [6], True), (64, 1, 128, [200, 64], [3, 20], False),         # few rows
    (16, 16, 64, [300] * 16, [250] * 16, True), (32, 16, 192, [64] * 17, [130] * 17, False)])
def test_attention_of_very_large_scores(ops, dtype, P, H, D, past, new, causal):
    """Scores from thousands to 1e30: the key that the queries point at, 127 of
    their signs everywhere, stands out by a factor of several, so that the
    output is its value, rounded once."""
    g = gen(92)
    cache, table = filled(g, P, H, D, past, new)
    sign = torch.randint(0, 2, (D,), generator=g, device="cuda") * 2 - 1
    # One key scale (a larger page scale could lift another key past this one).
    cache.k_scale.fill_(0.0123)
    first = table[:, 0].long()
    cache.k[first, :, 2] = (127 * sign).to(torch.int8)
    n = sum(new)
    gain = torch.exp(torch.linspace(math.log(1e4), math.log(1e30), n, device="cuda"))[:, None, None]
    q = (sign * gain).expand(n, H, D).to(dtype).contiguous()
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
    want = (cache.v[first, :, :, 2].double() * cache.v_scale[first].double()[..., None])[seq]
    # (The second term: other keys' probabilities, below 2^-1000, and the two roundings of p times scale.)
    assert ((o.double() - want).abs() <= (U[dtype] + 2.0 ** -20 + (0 if dtype == F32 else 2.0 ** -11)) * want.abs()).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("P,H,D,group,past,new,causal,window", [
    (32, 16, 64, 1, [250, 171, 33], [1, 1, 1], True, 0), (16, 4, 64, 1, [689, 500], [25, 19], True, 72),
    (64, 2, 128, 4, [8000, 900], [1, 1], True, 0), (16, 1, 96, 4, [100], [20], False, 0),
    (32, 2, 256, 1, [60], [80], True, 0)])
def test_attention_of_few_rows_is_rounded_once(ops, dtype, P, H, D, group, past, new, causal, window):
    """Up to 80 query rows a cache head: the probabilities hold two fp16 terms,
    so that the output's own rounding is nearly all of the error."""
    g = gen(93 + D)
    cache, table = filled(g, P, H, D, past, new)
    q = randn(g, sum(new), H * group, D, dtype=dtype)
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q, causal=causal, window=window)
    ref, tol = attend64_by_keys(cache, table, past, new, q, D ** -0.5, causal, window, two=True)
    worst = ((o.double() - ref).abs() / tol).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("M,N,K", [(15000, 8, 1), (40000, 8, 1), (40000, 8, 16)])
@pytest.mark.parametrize("spread", [0.01, 0.1, 0.5, 1.0, 2.0, 4.0])
def test_matmul_int_gelu_of_fp32(ops, M, N, K, spread):
    """GELU itself: one code of 1 and the inputs as the row's scale make the
    product exact.  0.5 x (1 + erf) in fp32 is within 1.8 units of |x| 2^-24;
    so is the kernels' form with an exact reciprocal and exponential, and a
    unit more in each of these, where erfc is at most 0.16, adds 0.4."""
    g = gen(95)
    a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    a[:, 0] = 1
    x = randn(g, M, std=spread)
    y = V.matmul_int(ops, a, x, a[:N].contiguous(), torch.ones(N, device="cuda"), gelu=True, dtype=F32)
    x = x.double()[:, None]
    err = (y.double() - 0.5 * x * torch.special.erfc(-x / math.sqrt(2))).abs()
    worst = (err / x.abs()).max().item() * 2 ** 24
    assert worst <= 2.2, worst
    # RMS: 0.5 x (1 + erf) has 3.8e-8 at a spread of 0.1 and less above 1.
    assert err.norm() <= 4.2e-8 * (N ** 0.5) * gelu64(x).norm()


# ---------------------------------------- attention's kernel for many rows
def check_kernel(ops, name, shape=None):
    got = V.voc_dbg_last_kernel(ops)
    assert got[0] == name and (shape is None or got[1] == shape), got


def close(o, ref, tol):
    worst = ((o.double() - ref).abs() / tol).max().item()
    assert worst <= 1, worst


MANY = [
    # P, kv heads, D, group, past, new, causal, window, parts (None: 1 or 2)
    (16, 16, 160, 1, [9 * i for i in range(16)], [130 - 3 * i for i in range(16)], True, 0, 1),
    (32, 16, 192, 1, [50] * 16, [99] * 16, True, 40, 1),
    (64, 8, 224, 2, [3 * i for i in range(32)], [41 + i % 7 for i in range(32)], False, 0, 1),
    (128, 16, 256, 1, [0] * 16, [128] * 16, True, 0, 1),
    (16, 4, 32, 3, [i for i in range(64)], [64] * 64, True, 0, 1),
    (64, 4, 128, 5, [200 - 3 * i for i in range(64)], [20] * 64, True, 0, 1),
    # Long enough for two parts of the keys, a short sequence among them.
    (16, 16, 160, 1, [1000, 7], [600, 333], True, 0, 2), (32, 16, 192, 1, [1000, 0], [599, 600], True, 0, 2),
    (64, 16, 224, 1, [1111, 40], [601, 1], True, 0, 2), (128, 16, 256, 1, [1000, 900], [600, 600], True, 0, 2),
    (16, 16, 96, 1, [1000, 1], [600, 577], True, 0, 2), (64, 16, 128, 1, [1005, 65], [600, 600], True, 0, 2),
    (32, 16, 64, 1, [1000, 0, 64, 999], [500, 500, 3, 450], True, 0, 2),
    (16, 16, 32, 1, [1000, 0, 64, 999], [500, 500, 3, 450], True, 0, 2),
    # Many parts.
    (64, 8, 128, 1, [7900], [256], False, 0, None), (32, 8, 256, 1, [8000], [257], False, 0, None),
    (128, 2, 192, 8, [16100], [70], True, 0, None),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,group,past,new,causal,window,parts", MANY)
def test_attention_of_many_rows(ops, dtype, P, H, D, group, past, new, causal, window, parts):
    g = gen(P + D + sum(past))
    cache, table = filled(g, P, H, D, past, new)
    q = randn(g, sum(new), H * group, D, dtype=dtype)
    b = batch_of(table, past, new)
    o = V.cache_attention(ops, cache, b, q, causal=causal, window=window)
    name, shape = V.voc_dbg_last_kernel(ops)
    assert name == "attend_many" and shape[0] == (128 if dtype == F32 or D > 128 else 256), (name, shape)
    assert shape[1] > 4 if parts is None else shape[1] == parts, shape
    close(o, *attend64(cache, table, past, new, q, D ** -0.5, causal, window))
    assert torch.equal(o, V.cache_attention(ops, cache, b, q, causal=causal, window=window))


# Few rows, many rows whole, many rows in two parts.
SIZES = [("attend_few", 32, 4, 64, [100, 61], [20, 3], 1), ("attend_many", 16, 16, 64, [40] * 16, [140] * 16, 1),
         ("attend_many", 64, 16, 192, [1000, 100], [600, 600], 2)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("kernel,P,H,D,past,new,parts", SIZES)
def test_attention_negative_scale_and_sharp_scores(ops, dtype, kernel, P, H, D, past, new, parts):
    g = gen(96)
    for spread, std, scale in ((1.0, 1.0, -0.15), (30.0, 4.0, D ** -0.5), (30.0, 4.0, -(D ** -0.5))):
        cache, table = filled(g, P, H, D, past, new, spread=spread)
        q = randn(g, sum(new), H, D, dtype=dtype, std=std)
        o = V.cache_attention(ops, cache, batch_of(table, past, new), q, scale=scale)
        check_kernel(ops, kernel, (V.voc_dbg_last_kernel(ops)[1][0], parts))
        close(o, *attend64_by_keys(cache, table, past, new, q, scale, True, 0))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("kernel,P,H,D,past,new,parts", SIZES)
def test_attention_missing_and_non_finite_pages(ops, dtype, kernel, P, H, D, past, new, parts):
    """Pages that are missing (also the first, the last and a whole block of 64
    keys), windows that lie in them, pages with NaN scales, a NaN query."""
    g = gen(97)
    cache, table = filled(g, P, H, D, past, new)
    q = randn(g, sum(new), H, D, dtype=dtype)
    last = (past[0] + new[0] - 1) // P
    block = [c for c in range(last) if c * P < 64 <= c * P + P or 64 <= c * P < 128]     # keys 64 .. 127 and some
    for columns in ([1], [0, last], block):
        hole = table.clone()
        for i, c in enumerate(columns):
            hole[0, c] = -1 if i % 2 else 1 << 30
        for window in (0, 3):
            out = torch.full_like(q, 7.0)
            V.cache_attention(ops, cache, batch_of(hole, past, new), q, window=window, out=out)
            ref, tol = attend64_by_keys(cache, table, past, new, q, D ** -0.5, True, window, hole=[(0, c) for c in columns])
            assert torch.equal((out == 0).all(-1), (ref == 0).all(-1))
            # (Windows of 3 keys give values beyond fp16 here: those round to infinity.)
            over = ref.to(dtype).isinf()
            assert torch.equal(out[over], ref.to(dtype)[over]) and ((out.double() - ref).abs() <= tol)[~over].all()
    o = V.cache_attention(ops, cache, batch_of(torch.full_like(table, -1), past, new), q, out=torch.full_like(q, 7.0))
    check_kernel(ops, kernel)
    assert (o == 0).all()
    ref, tol = attend64_by_keys(cache, table, past, new, q, D ** -0.5, True, 0)
    at = past[0] + torch.arange(new[0], device="cuda")
    for s in (cache.k_scale, cache.v_scale):
        kept, bad = s.clone(), torch.zeros(sum(new), H, dtype=torch.bool, device="cuda")
        for column, head in ((past[0] // P + 1, 1), (0, 2)):
            s[int(table[0, column]), head] = float("nan")
            bad[:new[0], head] |= at >= column * P
        o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
        assert o[bad].isnan().all() and ((o.double() - ref).abs() <= tol)[~bad].all()
        s.copy_(kept)
    q[5, 1, 3] = float("nan")
    o = V.cache_attention(ops, cache, batch_of(table, past, new), q)
    bad = torch.zeros(sum(new), H, dtype=torch.bool, device="cuda")
    bad[5, 1] = True
    assert o[bad].isnan().all() and ((o.double() - ref).abs() <= tol)[~bad].all()


@pytest.mark.parametrize("kernel,P,H,D,past,new,parts", SIZES)
def test_attention_strided_with_rows_between(ops, kernel, P, H, D, past, new, parts):
    g = gen(98)
    cache, table = filled(g, P, H, D, past, new)
    n = sum(new)
    big = randn(g, n + 5, 3, H, D, dtype=F16)
    q = big[:, 1]
    out = torch.full((n + 5, H, 2, D), 9.0, dtype=F16, device="cuda")[:, :, 0]
    starts = [2 + s for s in starts_of(new)]
    b = V.KVBatch(table, i32(past), i32(starts), max(new) + 6, 4096)
    V.cache_attention(ops, cache, b, q, out=out)
    check_kernel(ops, kernel)
    close(out[2:2 + n], *attend64(cache, table, past, new, q[2:2 + n], D ** -0.5, True, 0))
    assert (out[:2] == 9).all() and (out[2 + n:] == 9).all()


@pytest.mark.parametrize("kernel,P,H,D,past,new,parts", SIZES)
def test_attention_ranges_of_queries(ops, kernel, P, H, D, past, new, parts):
    """Rows of very large, very small and zero queries beside ordinary ones."""
    g = gen(99)
    cache, table = filled(g, P, H, D, past, new)
    n = sum(new)
    gain = torch.tensor([1e30, 1e-30, 0.0, 1.0, 1e-38, 1e4], device="cuda").repeat(-(-n // 6))[:n, None, None]
    for dtype in (F32, BF16):
        q = (randn(g, n, H, D) * gain).to(dtype)
        o = V.cache_attention(ops, cache, batch_of(table, past, new), q, scale=1e-3)
        check_kernel(ops, kernel)
        ref, tol = attend64_by_keys(cache, table, past, new, q, 1e-3, True, 0)
        # (Among scores of 1e28 ties cannot be told from near ties.)
        assert ((o.double() - ref).abs() <= tol)[gain[:, 0, 0] < 1e30].all()
        assert torch.isfinite(o).all()


def test_attention_of_many_rows_beyond_4_gib(ops):
    """The same offsets past 32 bits for the kernel for many rows."""
    g = gen(86)
    P, H, D, pages, n = 128, 8, 256, 17000, 2300
    cache = V.KVCache.from_tensors(
        torch.empty(pages, H, P, D, dtype=torch.int8, device="cuda"),
        torch.empty(pages, H, D, P, dtype=torch.int8, device="cuda"),
        torch.full((pages, H), float("nan"), device="cuda"), torch.full((pages, H), float("nan"), device="cuda"))
    table = torch.arange(pages - 18, pages, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
    k, v, q = (randn(g, n, H, D, dtype=F16) for _ in range(3))
    b = batch_of(table, [0], [n])
    V.cache_append(ops, cache, b, k, v)
    o = V.cache_attention(ops, cache, b, q)
    check_kernel(ops, "attend_many")
    close(o, *attend64(cache, table, [0], [n], q, 1 / 16, True, 0))


# ----------------------------------------------- every form of the product
def check_product_on_gpu(y, a, b, sa, sb, bias, gelu):
    """check_product with the integer sums in 64-bit floats (below 2^53) on the GPU."""
    prod = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    add = torch.zeros_like(sb, dtype=torch.float64) if bias is None else bias.double()
    ref, size = prod + add, prod.abs() + add.abs()
    err = 4 * E * size
    if gelu:
        err, ref = 1.13 * err + 8 * E * size, gelu64(ref)
    close(y, ref, err * (1 + U[y.dtype]) + U[y.dtype] * ref.abs() + SUB[y.dtype] + 1e-300)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,N,K,pad,offset,kernel,shape", [
    # Few tokens, 16, 32 and 64 a workgroup, rows that can be read as they lie.
    (3, 500, 200, 0, 0, "product_few", (16, 16)), (16, 4100, 64, 16, 0, "product_few", (16, 16)),
    (32, 4096, 1024, 0, 0, "product_few", (16, 32)), (17, 3100, 200, 0, 4, "product_few", (16, 32)),
    (33, 3100, 128, 0, 0, "product_few", (16, 64)), (64, 2000, 4096, 0, 0, "product_few", (16, 32)),
    (70, 1560, 1056, 4, 4, "product_few", (16, 64)),
    # Rows that are read in shifted words.
    (5, 1000, 333, 0, 1, "product_few_shifted", (16, 16)), (20, 3100, 333, 0, 3, "product_few_shifted", (16, 32)),
    (40, 3100, 77, 0, 0, "product_few_shifted", (16, 64)), (70, 2000, 333, 2, 5, "product_few_shifted", (16, 64)),
    (64, 3200, 1709, 0, 0, "product_few_shifted", (16, 64)), (1, 70, 3, 0, 1, "product_few_shifted", (16, 16)),
    # Every tile.
    (700, 640, 2064, 0, 0, "product_tile", (64, 64)), (390, 700, 16, 0, 0, "product_tile", (64, 64)),
    (2000, 1600, 208, 0, 16, "product_tile", (128, 64)), (2500, 2500, 400, 16, 0, "product_tile", (128, 128)),
    (3331, 3900, 272, 0, 0, "product_tile", (256, 256)), (1300, 1210, 77, 0, 0, "product_tile_rows", (64, 64)),
    (600, 700, 128, 8, 0, "product_tile_rows", (64, 64))])
def test_matmul_int_forms_with_bias_and_gelu(ops, dtype, M, N, K, pad, offset, kernel, shape):
    g = gen(M + N + K)

    def codes(rows):
        x = torch.randint(-127, 128, (rows * (K + pad) + offset,), generator=g, device="cuda", dtype=torch.int8)
        return x[offset:].view(rows, K + pad)[:, :K]

    a, b = codes(M), codes(N)
    sa = torch.rand(M, generator=g, device="cuda") * 0.02
    sb = torch.rand(N, generator=g, device="cuda") * 0.02 / math.sqrt(K)
    bias = randn(g, N)
    for use, gelu in ((bias, True), (bias, False), (None, True)):
        for width in (N, N + 3):                       # rows of outputs that are aligned and that are not
            big = torch.full((M + 1, width), 7.0, dtype=dtype, device="cuda")
            y = V.matmul_int(ops, a, sa, b, sb, bias=use, gelu=gelu, out=big[:M, :N])
            check_kernel(ops, kernel, shape)
            check_product_on_gpu(y, a, b, sa, sb, use, gelu)
            assert (big[M:] == 7).all() and (big[:, N:] == 7).all()


# ------------------------------------------------ every form of the append
def appended(cache, table, past, new, k, v):
    """What cache_append leaves, by the stated formulas in fp32 on the CPU:
    (codes [pages, H, P, D], scales) of keys and values."""
    inv127 = torch.tensor(1.0, dtype=F32) / 127
    P, out = cache.page_tokens, []
    starts = starts_of(new)
    for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v.transpose(2, 3), cache.v_scale, v)):
        codes, scale, x = codes.cpu().float(), scale.cpu().clone(), x.cpu().float()
        for b in range(len(past)):
            for t0 in range(past[b] // P * P, past[b] + new[b], P):
                page, lo, hi = int(table[b, t0 // P]), max(t0, past[b]), min(t0 + P, past[b] + new[b])
                rows = x[starts[b] + lo - past[b]:starts[b] + hi - past[b]].transpose(0, 1)      # [H, tokens, D]
                amax = rows.abs().amax((1, 2))
                own = torch.where(amax < 2.0 ** -100, torch.zeros(()), amax * inv127)
                was = scale[page].clone() if lo > t0 else torch.zeros_like(own)
                now = torch.maximum(was, own)
                inv = torch.where(now > 0, 1 / now, torch.zeros(()))[:, None, None]
                if lo > t0:
                    kept = codes[page][:, :lo - t0]
                    codes[page][:, :lo - t0] = torch.where((now > was)[:, None, None], (kept * (was[:, None, None] * inv)).round(), kept)
                codes[page][:, lo - t0:hi - t0] = (rows * inv).round().clamp(-127, 127)
                scale[page] = now
        out += [codes, scale]
    return out


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,past,new,lean,kernel,threads", [
    # Few tokens, into partly filled pages and over their ends.
    (16, 2, 64, [5, 15, 0], [1, 2, 8], 0, "append", 256), (64, 3, 96, [60, 63, 200], [8, 1, 5], 0, "append", 256),
    (128, 1, 256, [127, 3], [2, 7], 0, "append", 256),
    # Rows of any alignment, any number of tokens.
    (16, 2, 64, [5, 0], [40, 17], 1, "append", 256), (64, 3, 128, [100, 64], [9, 130], 3, "append", 256),
    (32, 1, 160, [31, 7], [200, 1], 1, "append", 256),
    # Pages built whole: one wave, where there are pages enough; two; four; more units than stay in registers.
    (16, 16, 64, [(7 * i) % 40 for i in range(40)], [40] * 40, 0, "append_page", 64),
    (16, 16, 128, [(5 * i) % 33 for i in range(40)], [40 - i % 9 for i in range(40)], 0, "append_page", 64),
    (32, 16, 64, [(9 * i) % 64 for i in range(48)], [33] * 48, 0, "append_page", 64),
    (32, 2, 64, [5, 31, 32, 0], [9, 70, 3, 64], 0, "append_page", 128), (128, 2, 32, [100, 0], [60, 9], 0, "append_page", 128),
    (16, 1, 224, [3, 0], [30, 16], 0, "append_page", 128),
    (64, 2, 128, [70, 3, 0], [25, 200, 64], 0, "append_page", 256), (128, 1, 256, [130, 1], [300, 127], 0, "append_page", 256),
    (64, 2, 192, [33, 63], [10, 66], 0, "append_page", 256)])
def test_append_follows_its_formulas(ops, dtype, P, H, D, past, new, lean, kernel, threads):
    """Codes and scales bit for bit, over pages that hold tokens: some heads'
    scales grow by the new tokens, some by far, some stay, one is all zeros."""
    g = gen(P + D + sum(new))
    table, pages = table_for(g, [-(-(p + n) // P) for p, n in zip(past, new)], spare=1)
    cache = V.KVCache(pages, P, H, D)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g, device="cuda", dtype=torch.int8))
        scale.copy_(torch.rand(scale.shape, generator=g, device="cuda") * 0.02 + 0.005)
    n, wide = sum(new), 2 * H * D + 8 * (1 if lean else 0)
    big = randn(g, n, wide, dtype=dtype)[:, lean:lean + 2 * H * D].view(n, 2 * H, D)
    gain = torch.tensor([1.0, 0.05, 30.0], device="cuda")[torch.arange(2 * H, device="cuda") % 3]
    big.mul_(gain[:, None].to(dtype))
    big[:, H + H // 2] = 0
    k, v = big[:, :H], big[:, H:]
    want = appended(cache, table, past, new, k, v)
    before = cache.k.clone(), cache.v.clone(), cache.k_scale.clone(), cache.v_scale.clone()
    V.cache_append(ops, cache, batch_of(table, past, new), k, v)
    check_kernel(ops, kernel, (threads, P))
    got = [cache.k.cpu().float(), cache.k_scale.cpu(), cache.v.transpose(2, 3).cpu().float(), cache.v_scale.cpu()]
    assert torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])
    touched = torch.zeros(pages, dtype=torch.bool, device="cuda")
    for b in range(len(past)):
        for c in range(past[b] // P, -(-(past[b] + new[b]) // P)):
            page, live = int(table[b, c]), min(P, past[b] + new[b] - c * P)
            touched[page] = True
            for i in (0, 2):
                assert torch.equal(got[i][page, :, :live], want[i][page, :, :live]), (b, c, i)
    for x, old in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(x[~touched], old[~touched])


# ------------------------------------------------------- memory and streams
def calls_on(ops, n):
    """name -> (inputs, call(inputs, stream) -> new outputs): every helper, its
    outputs and its inputs of sizes that nothing else in these tests has."""
    g = gen(120)
    cache, table = filled(g, 16, 8, 64, [30], [n])
    b = batch_of(table, [30], [n])
    w, codes, s = torch.ones(512, device="cuda"), torch.ones(512, 512, dtype=torch.int8, device="cuda"), torch.ones(512, device="cuda")
    rows = lambda *shape, dtype=F32: torch.ones(n, *shape, device="cuda", dtype=dtype)     # noqa: E731
    return {
        "rms_norm": (lambda: [rows(512), rows(512)], lambda x, t: V.rms_norm(ops, x[0], w, residual=x[1], stream=t)),
        "quantize_rows": (lambda: [rows(512)], lambda x, t: V.quantize_rows(ops, x[0], stream=t)),
        "matmul_int": (lambda: [rows(512, dtype=torch.int8), rows()], lambda x, t: [V.matmul_int(ops, *x, codes, s, stream=t)]),
        "cache_append": (lambda: [rows(8, 64), rows(8, 64)], lambda x, t: [V.cache_append(ops, cache, b, *x, stream=t)][:0]),
        "cache_attention": (lambda: [rows(8, 64)], lambda x, t: [V.cache_attention(ops, cache, b, x[0], stream=t)]),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["rms_norm", "quantize_rows", "matmul_int", "cache_append", "cache_attention"])
def test_explicit_stream_keeps_memory(ops, name, raw):
    """While a call is pending on an explicit stream, the memory that it reads
    and writes is not handed out again on the current one, and its outputs are
    no memory that pending work of the current stream may still use."""
    n = 4099
    make, call = calls_on(ops, n)[name]
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    want = [x.clone() for x in call(make(), None)]
    torch.cuda.synchronize()
    sizes = [(x.shape, x.dtype) for x in make() + want]
    torch.cuda.synchronize()
    # The allocator does hand out a freed block of a size again at once.
    for shape, dtype in sizes:
        t = torch.empty(shape, dtype=dtype, device="cuda")
        at = t.data_ptr()
        del t
        assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() == at
    # Blocks of the outputs' sizes that pending work of the current stream uses.
    x = make()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    busy = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    taken = {t.data_ptr() for t in busy}
    del busy
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)                     # about 0.1 s
    y = call(x, stream)
    assert not taken & {t.data_ptr() for t in y}
    held = {t.data_ptr() for t in x + list(y)}
    del x, y
    fresh = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(3)]
    pending = not s.query()
    assert not held & {t.data_ptr() for t in fresh}
    assert pending                                         # (else the above says nothing)
    # And what comes out is right, used on the current stream after the wait, freed there.
    x = make()
    s.wait_stream(torch.cuda.current_stream())
    y = call(x, stream)
    torch.cuda.current_stream().wait_stream(s)
    for got, right in zip(y, want):
        assert torch.equal(got, right)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("step", [1, 7, 9, 50])
def test_append_then_attend_step_by_step(ops, dtype, step):
    """Two sequences of 50 tokens in steps: after every append the cache holds
    what the formulas make of the cache before it, bit for bit, and every output
    is the attention over just that cache."""
    g = gen(83 + step)
    P, H, D, n = 16, 2, 64, 50
    table, pages = table_for(g, [4, 4])
    cache = V.KVCache(pages, P, H, D)
    q, k, v = (randn(g, 2, n, H, D, dtype=dtype) for _ in range(3))
    for t in range(0, n, step):
        m = min(step, n - t)
        past, new = [t, t], [m, m]
        rows = [x[:, t:t + m].reshape(2 * m, H, D) for x in (q, k, v)]
        want = appended(cache, table, past, new, rows[1], rows[2])
        b = batch_of(table, past, new)
        V.cache_append(ops, cache, b, rows[1], rows[2])
        assert torch.equal(cache.k_scale.cpu(), want[1]) and torch.equal(cache.v_scale.cpu(), want[3])
        for s in range(2):
            for c in range(-(-(t + m) // P)):
                page, live = int(table[s, c]), min(P, t + m - c * P)
                assert torch.equal(cache.k[page, :, :live].cpu().float(), want[0][page, :, :live])
                assert torch.equal(cache.v[page, :, :, :live].transpose(1, 2).cpu().float(), want[2][page, :, :live])
        close(V.cache_attention(ops, cache, b, rows[0]), *attend64(cache, table, past, new, rows[0], 0.125, True, 0))
