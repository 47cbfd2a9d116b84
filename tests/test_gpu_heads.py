"""Norm and rotation of query and key heads, the same on the way into the 8-bit
cache, and the cache read back, against plain 64-bit implementations.

u is the unit roundoff of a type (half a step, relative), E that of fp32.  A
normed value carries at most 13 E: the fp32 sum of a head's squares is 8
products in a lane and up to 6 rounds among them, 16 E at the most, halved by
the root; mean and eps 2 E, halved; the root 2 E; two products.  cos and sin
are off by at most 2 E (the fp32 remainder of a quarter turn 0.4 E, the
polynomials 1.5 E).  The rotation adds two roundings, so that a rotated value
is off by at most (13 + 2 + 2) E of |a| + |b|, which is taken as 20 E; without
a norm as 5 E."""
import ctypes

import pytest
import torch

from dac_vocoder_decoding_amd import vocoder as V
from test_gpu_ops import (BF16, E, F16, F32, SUB, U, batch_of, filled, gen, i32, page_scales, randn, starts_of, table_for,
                          values_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    h = V.open_ops(0)
    yield h
    torch.cuda.synchronize()
    V.voc_ops_destroy(h)


def frequencies(pairs):
    return (10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / max(pairs, 1))).float()


def turned64(x, weight, freq, position, adjacent, eps):
    """(y, size): the result in 64 bits and |a| + |b| of each value's pair."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    y, size = x.clone(), x.abs()
    n = 0 if freq is None else freq.numel()
    if n:
        angle = (position.double()[:, None] * freq.double())[:, None]
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
        xa, xb = x[..., a], x[..., b]
        y[..., a] = xa * angle.cos() - xb * angle.sin()
        y[..., b] = xb * angle.cos() + xa * angle.sin()
        size[..., a] = size[..., b] = xa.abs() + xb.abs()
    return y, size


def check_turned(got, x, weight, freq, position, adjacent, eps):
    y, size = turned64(x, weight, freq, position, adjacent, eps)
    tol = (20 if weight is not None else 5) * E * size * (1 + U[x.dtype]) + U[x.dtype] * y.abs() + SUB[x.dtype]
    if freq is not None and freq.numel():
        # The angle itself is a product of 64 bits on both sides.
        tol = tol + 2.0 ** -50 * position.double().abs()[:, None, None] * freq.max().double() * size
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), ((got.double() - y).abs() / tol).max()


SHAPES = [
    # tokens, heads, kv heads, dim, pairs, first position
    (1, 1, 0, 2, 1, 0), (1, 1, 1, 64, 32, 5), (32, 16, 16, 64, 32, 225), (7, 5, 1, 128, 64, 1000000), (3, 2, 2, 256, 128, 77),
    (5, 3, 1, 96, 48, 0), (9, 4, 4, 80, 10, 300000), (4, 2, 1, 80, 20, 3), (6, 3, 3, 32, 4, 9), (2, 7, 2, 192, 96, 0),
    (5, 2, 1, 33, 5, 12), (3, 1, 1, 255, 127, 40), (2, 2, 1, 256, 127, 5), (4, 2, 2, 1, 0, 0), (3, 3, 1, 64, 0, 0),
    (300, 32, 8, 128, 64, 65000), (5000, 3, 1, 64, 16, 0)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,pairs,first", SHAPES)
def test_norm_rotate(ops, dtype, adjacent, tokens, heads, kv_heads, dim, pairs, first):
    g = gen(tokens + dim + pairs)
    qkv = randn(g, tokens, heads + 2 * kv_heads, dim, dtype=dtype, std=3.0)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads] if kv_heads else None
    kept = qkv.clone()
    qw, kw = 1 + randn(g, dim, std=0.3), 1 + randn(g, dim, std=0.3)
    freq = frequencies(pairs) if pairs else None
    position = torch.randperm(tokens, generator=g, device="cuda").to(torch.int32) + first
    for weights in ((qw, kw), (None, kw), (None, None)):
        args = dict(position=position, freq=freq, q_weight=weights[0], k_weight=weights[1], eps=1e-5, adjacent=adjacent)
        qo, ko = V.norm_rotate(ops, q, k, **args)
        assert (ko is None) == (k is None) and torch.equal(qkv, kept)
        check_turned(qo, q, weights[0], freq, position, adjacent, 1e-5)
        if k is not None:
            check_turned(ko, k, weights[1], freq, position, adjacent, 1e-5)
    # In place, the same bits; what lies between stays.
    V.norm_rotate(ops, q, k, q_out=q, k_out=k, **args)
    assert torch.equal(q, qo) and torch.equal(qkv[:, heads + kv_heads:], kept[:, heads + kv_heads:])
    assert k is None or torch.equal(k, ko)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,pairs,adjacent", [(64, 32, True), (64, 32, False), (128, 16, False), (96, 24, True), (80, 10, False)])
def test_norm_rotate_at_any_alignment(ops, dtype, dim, pairs, adjacent):
    """Rows that start at odd elements: the same bits as whole words."""
    g = gen(dim + pairs)
    n, H = 9, 3
    position, freq, w = torch.arange(100, 100 + n, dtype=torch.int32, device="cuda"), frequencies(pairs), 1 + randn(g, dim, std=0.2)
    x = randn(g, n, H, dim, dtype=dtype)
    want, _ = V.norm_rotate(ops, x, position=position, freq=freq, q_weight=w, adjacent=adjacent)
    wide = torch.full((n * (H * dim + 7) + 9,), 7.0, dtype=dtype, device="cuda")
    odd = wide[3:3 + n * (H * dim + 7)].view(n, H * dim + 7)[:, :H * dim].view(n, H, dim)
    odd.copy_(x)
    out = torch.full_like(wide, 7.0)
    got = out[1:1 + n * (H * dim + 7)].view(n, H * dim + 7)[:, :H * dim].view(n, H, dim)
    V.norm_rotate(ops, odd, position=position, freq=freq, q_weight=w, adjacent=adjacent, q_out=got)
    assert V.voc_dbg_last_kernel(ops)[1][1] == 2
    assert torch.equal(got, want)
    left = out.clone()
    left[1:1 + n * (H * dim + 7)].view(n, H * dim + 7)[:, :H * dim].fill_(7.0)
    assert (left == 7).all()


def test_norm_rotate_positions_and_empty(ops):
    """Negative positions turn back, the largest keep their angles; no tokens."""
    g = gen(2)
    x, freq = randn(g, 4, 2, 64), frequencies(32)
    position = i32([0, -5, 2 ** 31 - 1, -2 ** 31])
    y, _ = V.norm_rotate(ops, x, position=position, freq=freq, adjacent=True)
    assert torch.equal(y[0], x[0])
    check_turned(y, x, None, freq, position, True, 0)
    back, _ = V.norm_rotate(ops, y[1:2], position=i32([5]), freq=freq, adjacent=True)
    assert (back - x[1:2]).abs().max() <= 16 * E * x.abs().max()       # two turns of 5 E of |a| + |b|
    empty, none = V.norm_rotate(ops, x[:0], x[:0], position=position[:0], freq=freq)
    assert empty.shape == (0, 2, 64) and none.shape == (0, 2, 64)
    same, _ = V.norm_rotate(ops, x)
    assert torch.equal(same, x)


@pytest.mark.parametrize("adjacent", [False, True])
def test_norm_rotate_non_finite(ops, adjacent):
    """A head that is not finite, or whose squares pass fp32, becomes NaN, its
    neighbours do not; a head of zeros stays one."""
    g = gen(3)
    x = randn(g, 3, 4, 64)
    x[0, 1, 5], x[1, 2, 60], x[2, 0] = float("nan"), float("inf"), 0
    x[2, 3] = 1e25
    position, freq, w = i32([3, 4, 5]), frequencies(16), torch.ones(64, device="cuda")
    y, _ = V.norm_rotate(ops, x, position=position, freq=freq, q_weight=w, adjacent=adjacent)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = bad[2, 3] = True
    assert y[bad].isnan().all() and y[~bad].isfinite().all() and not y[2, 0].any()
    # Without a norm a value that is not finite touches its own pair only.
    y, _ = V.norm_rotate(ops, x, position=position, freq=freq, adjacent=adjacent)
    assert (~y[1, 2].isfinite()).sum() == 1 and (~y[0, 1].isfinite()).sum() == 2


# ---------------------------------------------------------- into the cache
def cache_and_rows(g, P, H, D, group, past, new, dtype, pad=0):
    """A cache that holds the past (its idle pages NaN), its table, and the rows
    of queries, keys and values."""
    cache, table = filled(g, P, H, D, past, [0] * len(past))
    spare = [-(-(p + n) // P) + 1 for p, n in zip(past, new)]
    table, pages = table_for(g, spare)
    cache = V.KVCache(pages, P, H, D)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g, device="cuda", dtype=torch.int8))
        scale.copy_(torch.rand(scale.shape, generator=g, device="cuda") * 0.02 + 0.005)
        for b, p in enumerate(past):
            scale[table[b, -(-p // P):spare[b]].long()] = float("nan")
    n, heads = sum(new), H * (group + 2)
    rows = randn(g, n, heads * D + pad, dtype=dtype, std=1.5)[:, pad:].view(n, heads, D)
    gain = torch.tensor([1.0, 0.05, 30.0], device="cuda")[torch.arange(heads, device="cuda") % 3].to(dtype)
    rows.mul_(gain[:, None])
    return cache, table, rows[:, :H * group], rows[:, H * group:H * (group + 1)], rows[:, H * (group + 1):]


def copy_of(cache):
    return V.KVCache.from_tensors(*(t.clone() for t in cache.tensors))


def positions(past, new):
    return torch.cat([torch.arange(p, p + n, dtype=torch.int32, device="cuda") for p, n in zip(past, new)])


STEPS = [
    # page, kv heads, dim, query heads to one, past, new
    (16, 2, 64, 1, [25, 0, 15, 16], [1, 1, 1, 1]), (64, 8, 128, 4, [100, 63], [1, 1]), (16, 1, 32, 3, [3], [8]),
    (32, 3, 96, 1, [31, 0, 7], [2, 5, 33]), (16, 16, 64, 1, [100] * 6, [25] * 6), (64, 2, 128, 4, [0, 70, 5], [200, 25, 0]),
    (128, 1, 256, 2, [130, 1], [300, 127]), (16, 2, 256, 1, [0], [40]), (128, 2, 32, 1, [100, 0], [60, 300]),
    (32, 1, 192, 5, [7, 31], [1, 70]), (16, 5, 160, 1, [0, 17], [16, 15]), (64, 4, 64, 2, [9], [1000]),
    (32, 16, 64, 1, [(9 * i) % 64 for i in range(48)], [33] * 48), (128, 8, 128, 1, [77, 0], [700, 650]),
    (16, 1, 224, 1, [3, 0], [30, 16])]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("P,H,D,group,past,new", STEPS)
def test_append_of_heads_as_they_are(ops, dtype, pad, P, H, D, group, past, new):
    """Without norm and rotation: the cache of cache_append bit for bit, the
    queries unchanged."""
    g = gen(P + D + sum(new))
    cache, table, q, k, v = cache_and_rows(g, P, H, D, group, past, new, dtype, pad)
    plain, b = copy_of(cache), batch_of(table, past, new)
    V.cache_append(ops, plain, b, k, v)
    out = V.norm_rotate_append(ops, cache, b, q, k, v)
    assert torch.equal(out, q)
    used = torch.zeros(cache.k.shape[0], dtype=torch.bool, device="cuda")
    for s, (p, n) in enumerate(zip(past, new)):
        for c in range(p // P, -(-(p + n) // P)):
            page, live = int(table[s, c]), min(P, p + n - c * P)
            used[page] = True
            assert torch.equal(cache.k[page, :, :live], plain.k[page, :, :live])
            assert torch.equal(cache.v[page, ..., :live], plain.v[page, ..., :live])
            assert torch.equal(cache.k_scale[page], plain.k_scale[page]) and torch.equal(cache.v_scale[page], plain.v_scale[page])
    assert torch.equal(cache.k[~used], plain.k[~used]) and torch.equal(cache.v[~used], plain.v[~used])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("adjacent,part", [(True, 1.0), (False, 1.0), (False, 0.5), (True, 0.3)])
@pytest.mark.parametrize("P,H,D,group,past,new", STEPS)
def test_norm_rotate_append(ops, dtype, adjacent, part, P, H, D, group, past, new):
    """Queries as norm_rotate leaves them; values as cache_append does; keys
    within half a step of the normed and rotated ones, their page's scale the
    largest of them or the older scale."""
    g = gen(P * 3 + D + sum(new))
    cache, table, q, k, v = cache_and_rows(g, P, H, D, group, past, new, dtype)
    pairs = int(D // 2 * part)
    freq, qw, kw = frequencies(pairs), 1 + randn(g, D, std=0.3), 1 + randn(g, D, std=0.3)
    plain, b, pos = copy_of(cache), batch_of(table, past, new), positions(past, new)
    olds = [values_of(cache, table, s, p, "k") for s, p in enumerate(past)]
    before = copy_of(cache)
    V.cache_append(ops, plain, b, k, v)
    args = dict(freq=freq, q_weight=qw, k_weight=kw, eps=1e-5, adjacent=adjacent)
    out = V.norm_rotate_append(ops, cache, b, q, k, v, **args)
    check_turned(out, q, qw, freq, pos, adjacent, 1e-5)
    assert torch.equal(out, V.norm_rotate(ops, q, position=pos, freq=freq, q_weight=qw, eps=1e-5, adjacent=adjacent)[0])
    want, _ = turned64(k, kw, freq, pos, adjacent, 1e-5)
    at, used = 0, torch.zeros(cache.k.shape[0], dtype=torch.bool, device="cuda")
    for s, (p, n) in enumerate(zip(past, new)):
        if not n:
            continue
        x = want[at:at + n].transpose(0, 1)                                    # [H, n, D]
        at += n
        got, scale = values_of(cache, table, s, p + n, "k"), page_scales(cache, table, s, p + n, "k")
        # A rotated value's error of 20 E (|a| + |b|) is at most 40 E of the
        # pair's larger result; the hardware's sine and the like may serve codes
        # of 7 bits: 2^-18 of a pair is what is asked of them here.
        rel = 40 * E + 2.0 ** -18
        tol = scale[..., None] * (0.5 + 127 * (2 * rel + 6 * E))
        assert ((got[:, p:] - x).abs() <= tol[:, p:]).all()
        assert ((got[:, :p] - olds[s]).abs() <= tol[:, :p])[:, p // P * P:].all()
        assert torch.equal(got[:, :p // P * P], olds[s][:, :p // P * P])
        for c in range(p // P, -(-(p + n) // P)):
            page, lo, hi = int(table[s, c]), max(c * P, p), min(c * P + P, p + n)
            used[page] = True
            own = x[:, lo - p:hi - p].abs().amax((1, 2)) / 127
            older = before.k_scale[page].double() if lo > c * P else torch.zeros_like(own)
            now = torch.maximum(own, older)
            assert ((cache.k_scale[page].double() - now).abs() <= (rel + 3 * E) * now).all()
            assert torch.equal(cache.v[page, ..., :hi - c * P], plain.v[page, ..., :hi - c * P])
            assert torch.equal(cache.v_scale[page], plain.v_scale[page])
    assert torch.equal(cache.k[~used], before.k[~used]) and torch.equal(cache.v[~used], before.v[~used])
    # Queries in place, or none at all: the same cache.
    again = copy_of(before)
    mine = q.clone()
    assert V.norm_rotate_append(ops, again, b, mine, k, v, out=mine, **args) is mine and torch.equal(mine, out)
    only = copy_of(before)
    assert V.norm_rotate_append(ops, only, b, None, k, v, **args) is None
    for x, y, z in zip(cache.tensors, again.tensors, only.tensors):
        assert torch.equal(x.nan_to_num(7), y.nan_to_num(7)) and torch.equal(x.nan_to_num(7), z.nan_to_num(7))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("n", [3, 40])
def test_norm_rotate_append_non_finite(ops, dtype, n):
    """A key head that is not finite makes its page's scale NaN, of that head."""
    g = gen(8)
    P, H, D = 16, 3, 64
    table, pages = table_for(g, [-(-n // P)])
    cache = V.KVCache(pages, P, H, D)
    k = randn(g, n, H, D, dtype=dtype)
    k[:, 1] = 0
    k[2, 2, 5] = float("nan")
    k[n - 1, 0, 1] = float("inf")
    V.norm_rotate_append(ops, cache, batch_of(table, [0], [n]), k, k, torch.ones_like(k), freq=frequencies(32),
                         k_weight=torch.ones(D, device="cuda"))
    first, last = int(table[0, 0]), int(table[0, (n - 1) // P])
    assert cache.k_scale[first, 2].isnan() and cache.k_scale[last, 0].isnan() and not cache.k[first, 2, :min(n, P)].any()
    assert cache.k_scale[first, 1] == 0 and not cache.k[first, 1, :min(n, P)].any()
    assert (n <= P or cache.k_scale[first, 0] > 0) and cache.v_scale[first].isfinite().all()


@pytest.mark.parametrize("n", [2, 30])
def test_steps_stay_inside_the_table(ops, n):
    """Positions past the table, pages out of range and sequences whose rows are
    out of bounds leave the cache and every row as they are; queries of a
    sequence with rows are turned all the same."""
    g = gen(11)
    P, H, D = 16, 2, 64
    cache = V.KVCache(4, P, H, D)
    cache.k.fill_(5)
    cache.v.fill_(6)
    x = randn(g, 3 * n, H, D)
    table = i32([[0, 7], [-1, 1], [2, 3]])
    starts = i32([0, n, n + 5, 3 * n + 9])         # the last sequence's rows end past the rows
    b = V.KVBatch(table, i32([2 * P, 0, 0]), starts, max(n, 5), 2 * P + n)
    out = torch.full_like(x, 9.0)
    if n > 5:
        V.norm_rotate_append(ops, cache, b, x, x, x, freq=frequencies(32), out=out)
    else:
        b = V.KVBatch(table, i32([2 * P, 0, 0]), i32([0, n, n + 1, 3 * n + 9]), n, 2 * P + n)
        V.norm_rotate_append(ops, cache, b, x, x, x, freq=frequencies(32), out=out)
    rows = n + 5 if n > 5 else n + 1
    assert (cache.k == 5).all() and (cache.v == 6).all() and not cache.k_scale.any()
    assert (out[rows:] == 9).all() and (out[:rows] != 9).any(-1).all()
    k, v = torch.full_like(x, 8.0), torch.full_like(x, 8.0)
    V.cache_read(ops, cache, b, 3 * n, k=k, v=v)
    assert (k == 8).all() and (v == 8).all()


# ------------------------------------------------------------- read back
READS = [
    (16, 2, 64, [0, 5], [1, 40]), (64, 8, 128, [100, 0, 63], [25, 200, 1]), (128, 1, 256, [5], [300]), (16, 1, 32, [15], [2]),
    (32, 3, 96, [31, 0, 32], [1, 1, 100]), (16, 16, 64, [0] * 5, [250, 3, 0, 77, 16]), (128, 3, 160, [1], [127])]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,past,new", READS)
def test_cache_read(ops, dtype, P, H, D, past, new):
    """Code times scale in fp32, rounded once, bit for bit; strided outputs, rows
    of no sequence, one of the two alone."""
    g = gen(P + H + D)
    cache, table = filled(g, P, H, D, past, new)
    n, b = sum(new), batch_of(table, past, new)
    k, v = V.cache_read(ops, cache, b, n, dtype=dtype)

    def rows(codes, scale):
        out = []
        for s, (p, m) in enumerate(zip(past, new)):
            ids = table[s, :-(-(p + m) // P)].long()
            x = (codes[ids].float() * scale[ids][..., None, None]).to(dtype)   # [pages, H, P, D]
            out.append(x.transpose(1, 2).reshape(-1, H, D)[p:p + m])
        return torch.cat(out)

    want_k, want_v = rows(cache.k, cache.k_scale), rows(cache.v.transpose(2, 3), cache.v_scale)
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    for pad in (0, 8, 3):
        wide = torch.full((n + 2, 2 * H * D + pad), 7.0, dtype=dtype, device="cuda")
        both = wide[:, pad:].unflatten(1, (2 * H, D))
        assert both.data_ptr() == wide.data_ptr() + pad * wide.element_size()
        V.cache_read(ops, cache, b, n, k=both[:n, :H], v=both[:n, H:])
        assert torch.equal(both[:n, :H], want_k) and torch.equal(both[:n, H:], want_v)
        assert (wide[n:] == 7).all() and (wide[:, :pad] == 7).all()
    L, c = V.lib(), V._with_tokens(b, n)
    for which in (0, 1):
        one = torch.full((n, H, D), 7.0, dtype=dtype, device="cuda")
        ptr = [None, None]
        ptr[which] = one.data_ptr()
        assert L.vocoder_cache_read(ops, cache.ref, ctypes.byref(c), V._dtype(dtype), ptr[0], H * D, D, ptr[1], H * D, D,
                                    V._raw_stream(0)) == V.VOC_OK
        assert torch.equal(one, (want_k, want_v)[which])


def test_cache_read_non_finite_scales(ops):
    g = gen(5)
    cache, table = filled(g, 16, 2, 32, [0], [40])
    cache.k_scale[int(table[0, 1]), 1] = float("nan")
    k, v = V.cache_read(ops, cache, batch_of(table, [0], [40]), 40)
    assert k[16:32, 1].isnan().all() and k[:16].isfinite().all() and k[32:].isfinite().all() and k[:, 0].isfinite().all()
    assert v.isfinite().all()


def test_steps_and_reads_beyond_4_gib(ops):
    """Pages whose codes lie past 32-bit byte offsets."""
    g = gen(85)
    P, H, D, pages, n = 128, 8, 256, 17000, 300
    cache = V.KVCache.from_tensors(
        torch.empty(pages, H, P, D, dtype=torch.int8, device="cuda"), torch.empty(pages, H, D, P, dtype=torch.int8, device="cuda"),
        torch.full((pages, H), float("nan"), device="cuda"), torch.full((pages, H), float("nan"), device="cuda"))
    used = -(-n // P)
    table = torch.arange(pages - used, pages, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
    k, v, freq, w = randn(g, n, H, D, dtype=F16), randn(g, n, H, D, dtype=F16), frequencies(128), torch.ones(256, device="cuda")
    for past, new in (([0], [n - 1]), ([n - 1], [1])):
        rows = slice(past[0], past[0] + new[0])
        V.norm_rotate_append(ops, cache, batch_of(table, past, new), None, k[rows], v[rows], freq=freq, k_weight=w, eps=0.0)
    got_k, got_v = V.cache_read(ops, cache, batch_of(table, [0], [n]), n, dtype=F32)
    want, _ = turned64(k, w, freq, positions([0], [n]), False, 0.0)
    # Half a step, another where a scale grew with the last token.
    for got, x, which in ((got_k, want, "k"), (got_v, v.double(), "v")):
        step = page_scales(cache, table, 0, n, which).t()[..., None]
        assert ((got.double() - x).abs() <= step * (1.0 + 127 * (80 * E + 2.0 ** -17))).all()


def test_outputs_beyond_32_bit_offsets(ops):
    """Rows whose element offsets pass 2^31 (strided far apart)."""
    g = gen(6)
    n, H, D = 3, 2, 64
    stride = 1 << 30
    big = torch.empty(2 * stride + 2 * H * D, dtype=F16, device="cuda")
    far = big.as_strided((n, H, D), (stride, D, 1))
    x = randn(g, n, H, D, dtype=F16)
    position, freq = i32([1, 2, 3]), frequencies(32)
    want, _ = V.norm_rotate(ops, x, position=position, freq=freq)
    V.norm_rotate(ops, x, position=position, freq=freq, q_out=far)
    assert torch.equal(far, want)
    cache, table = filled(g, 16, H, D, [0], [n])
    k, v = V.cache_read(ops, cache, batch_of(table, [0], [n]), n)
    V.cache_read(ops, cache, batch_of(table, [0], [n]), n, k=far, v=far)
    other = V.cache_read(ops, cache, batch_of(table, [0], [n]), n, k=far)[1]
    assert torch.equal(far, k) and torch.equal(other, v)


# ----------------------------------------------------- streams and graphs
def test_steps_captured_and_replayed(ops):
    """A frame's norm, rotation, append, attention and read captured once and
    replayed on new rows and positions, eager calls between the replays."""
    g = gen(84)
    H, group, D, P, B, most = 2, 2, 64, 16, 3, 400
    table, pages = table_for(g, [-(-most // P)] * B)
    caches = [V.KVCache(pages, P, H, D) for _ in range(2)]
    past, starts = torch.zeros(B, dtype=torch.int32, device="cuda"), i32([0, 1, 2, 3])
    rows = randn(g, B, H * (group + 2), D, dtype=F16)
    freq, qw, kw = frequencies(32), 1 + randn(g, D, std=0.2), 1 + randn(g, D, std=0.2)

    def step(cache):
        b = V.KVBatch(table, past, starts, 1, most)
        q = V.norm_rotate_append(ops, cache, b, rows[:, :H * group], rows[:, H * group:-H], rows[:, -H:], freq=freq,
                                 q_weight=qw, k_weight=kw, adjacent=True)
        o = V.cache_attention(ops, cache, b, q)
        return (q, o, *V.cache_read(ops, cache, b, B), *V.norm_rotate(ops, o, position=past, freq=freq)[:1]), b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, keep0 = step(V.KVCache(pages, P, H, D))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, keep = step(caches[0])
    for t in range(20):
        rows.copy_(randn(g, *rows.shape, dtype=F16))
        past.fill_(t * 19)
        graph.replay()
        want, _ = step(caches[1])
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), t
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v_scale, caches[1].v_scale), t


def test_heads_refusals(ops):
    L = V.lib()
    x, w = torch.zeros(4, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    pos = i32([0, 1, 2, 3])

    def turn(dtype=0, tokens=4, dim=64, position=pos.data_ptr(), freq=w.data_ptr(), pairs=32, adjacent=0, eps=1e-6, heads=2,
             q=x.data_ptr(), qt=128, qh=64, qw=w.data_ptr(), qo=x.data_ptr(), ot=128, oh=64, kv=0, k=None, kt=0, kh=0, kw=None,
             ko=None, kot=0, koh=0):
        return L.vocoder_norm_rotate(ops, dtype, tokens, dim, position, freq, pairs, adjacent, eps, heads, q, qt, qh, qw, qo, ot,
                                     oh, kv, k, kt, kh, kw, ko, kot, koh, None)

    for kw in (dict(dtype=3), dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(dim=0), dict(dim=257), dict(position=None),
               dict(freq=None), dict(pairs=33), dict(pairs=-1), dict(pairs=2 ** 31 - 1), dict(adjacent=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(heads=-1), dict(heads=4097), dict(q=None), dict(qt=-1), dict(qh=1 << 41), dict(qw=w.data_ptr() + 2),
               dict(qo=None), dict(ot=-4), dict(oh=-1), dict(kv=1), dict(kv=1, k=x.data_ptr()), dict(kv=-1),
               dict(q=x.data_ptr() + 2), dict(freq=w.data_ptr() + 1), dict(position=pos.data_ptr() + 2)):
        assert turn(**kw) == V.VOC_INVALID_PARAMS, kw
        assert V.voc_ops_last_error(ops), kw
    assert turn(tokens=0, q=None) == V.VOC_OK and turn(heads=0, q=None, qo=None) == V.VOC_OK and V.voc_ops_last_error(ops) == ""

    cache = V.KVCache(4, 16, 2, 64)
    b = V.KVBatch(i32([[0, 1]]), i32([0]), i32([0, 1]), 1, 1)

    def step(dtype=0, freq=w.data_ptr(), pairs=32, adjacent=0, eps=1e-6, heads=2, q=x.data_ptr(), qt=128, qo=x.data_ptr(), k=x.data_ptr(),
             kt=128, kw=None, v=x.data_ptr(), vt=128, vh=64, **fields):
        c, n = V.voc_kv_cache(), V.voc_kv_batch()
        ctypes.pointer(c)[0], ctypes.pointer(n)[0] = cache.c, V._with_tokens(b, 1)
        for name, value in fields.items():
            setattr(c if hasattr(c, name) else n, name, value)
        return L.vocoder_norm_rotate_append(ops, ctypes.byref(c), ctypes.byref(n), dtype, freq, pairs, adjacent, eps, heads, q, qt,
                                            64, None, qo, 128, 64, k, kt, 64, kw, v, vt, vh, None)

    for kw in (dict(dtype=4), dict(freq=None), dict(pairs=33), dict(adjacent=-1), dict(eps=float("inf")), dict(heads=-1),
               dict(heads=5000), dict(q=None), dict(qt=-1), dict(qo=None), dict(k=None), dict(kt=-1), dict(v=None), dict(vt=-1),
               dict(vh=1 << 41), dict(kw=w.data_ptr() + 1), dict(page_tokens=8), dict(head_dim=48), dict(kv_heads=0),
               dict(n_pages=0), dict(batch=-1), dict(batch=70000), dict(table_stride=0), dict(starts=None), dict(past=None),
               dict(batch=65535, max_new=1 << 14)):
        assert step(**kw) == V.VOC_INVALID_PARAMS, kw
        assert V.voc_ops_last_error(ops), kw
    for kw in (dict(batch=0), dict(tokens=0), dict(max_new=0)):
        assert step(**kw) == V.VOC_OK

    def read(dtype=0, k=x.data_ptr(), kt=128, v=x.data_ptr(), vt=128, **fields):
        c, n = V.voc_kv_cache(), V.voc_kv_batch()
        ctypes.pointer(c)[0], ctypes.pointer(n)[0] = cache.c, V._with_tokens(b, 1)
        for name, value in fields.items():
            setattr(c if hasattr(c, name) else n, name, value)
        return L.vocoder_cache_read(ops, ctypes.byref(c), ctypes.byref(n), dtype, k, kt, 64, v, vt, 64, None)

    for kw in (dict(dtype=9), dict(kt=-1), dict(vt=-2), dict(k=x.data_ptr() + 2), dict(page_tokens=24), dict(past=None),
               dict(batch=65535, max_new=1 << 14)):
        assert read(**kw) == V.VOC_INVALID_PARAMS, kw
        assert V.voc_ops_last_error(ops), kw
    assert read(k=None, v=None, kt=-1) == V.VOC_OK and read(tokens=0) == V.VOC_OK
