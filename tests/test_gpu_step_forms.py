"""Every form of the step into the cache and of its read, by name, memory on
explicit streams, and several handles at once.  Bounds as in test_gpu_heads."""
import threading

import pytest
import torch

from dac_vocoder_decoding_amd import vocoder as V
from test_gpu_heads import cache_and_rows, check_turned, copy_of, frequencies, positions, turned64
from test_gpu_ops import BF16, E, F16, F32, batch_of, filled, gen, i32, randn, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    h = V.open_ops(0)
    yield h
    torch.cuda.synchronize()
    V.voc_ops_destroy(h)


def held(cache, table, past, new, which):
    """Keys or values of the new tokens [tokens, H, D] in 64 bits, and their page's scale."""
    P = cache.page_tokens
    at = torch.cat([torch.arange(p, p + n) for p, n in zip(past, new)]).cuda()
    b = torch.cat([torch.full((n,), s) for s, n in enumerate(new)]).cuda()
    page, slot = table[b, at // P].long(), at % P
    scale = (cache.k_scale if which == "k" else cache.v_scale)[page].double()[..., None]
    x = cache.k[page, :, slot] if which == "k" else cache.v[page, :, :, slot]
    return x.double() * scale, scale


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,group,past,new,adjacent,kernel,shape", [
    (16, 3, 32, 1, [7, 0], [20, 9], True, "step_page", (1, 1)), (16, 5, 64, 2, [3, 16], [30, 1], False, "step_page", (1, 2)),
    (32, 7, 64, 1, [31, 0], [40, 33], True, "step_page", (1, 4)), (16, 2, 128, 4, [1], [50], False, "step_page", (1, 4)),
    (64, 3, 64, 1, [60, 5], [9, 128], True, "step_page", (2, 4)), (128, 3, 32, 1, [100], [200], False, "step_page", (2, 4)),
    (32, 3, 96, 1, [9], [100], True, "step_page", (2, 4)), (64, 3, 128, 4, [63, 0], [10, 64], False, "step_page", (4, 4)),
    (32, 1, 160, 2, [30], [29], True, "step_page", (4, 4)), (128, 3, 128, 1, [127, 0], [130, 256], True, "step_page", (4, 8)),
    (64, 2, 256, 1, [5], [70], False, "step_page", (4, 8)), (128, 2, 256, 2, [100], [300], False, "step_page", (8, 8)),
    (16, 2, 64, 1, [5], [1], True, "step_page", (1, 2)), (64, 1, 128, 4, [60], [12], False, "step", (16, 1)),
    (64, 2, 64, 1, [60, 3], [1, 2], True, "step", (8, 0)), (128, 3, 256, 1, [127, 3, 0], [1, 5, 12], False, "step", (32, 1)),
    (32, 1, 64, 3, [31, 32], [2, 1], False, "step_page", (1, 4)),
    # Enough pages for several heads a workgroup, some groups short of a head; tokens in runs.
    (64, 5, 128, 1, [3 * i for i in range(7)], [4000 - 31 * i for i in range(7)], False, "step_page", (4, 4)),
    (16, 9, 64, 1, [i for i in range(60)], [500 - 7 * i for i in range(60)], True, "step_page", (1, 2))])
def test_step_forms(ops, dtype, P, H, D, group, past, new, adjacent, kernel, shape):
    g = gen(P + H + D)
    cache, table, q, k, v = cache_and_rows(g, P, H, D, group, past, new, dtype)
    freq, qw, kw, pos = frequencies(D // 2), 1 + randn(g, D, std=0.3), 1 + randn(g, D, std=0.3), positions(past, new)
    plain, b = copy_of(cache), batch_of(table, past, new)
    out = V.norm_rotate_append(ops, cache, b, q, k, v, freq=freq, q_weight=qw, k_weight=kw, eps=1e-5, adjacent=adjacent)
    assert V.voc_dbg_last_kernel(ops) == (kernel, shape)
    check_turned(out, q, qw, freq, pos, adjacent, 1e-5)
    want, _ = turned64(k, kw, freq, pos, adjacent, 1e-5)
    got, scale = held(cache, table, past, new, "k")
    assert ((got - want).abs() <= scale * (0.5 + 127 * (2 * (40 * E + 2.0 ** -18) + 6 * E))).all()
    V.cache_append(ops, plain, b, k, v)
    for s, (p, n) in enumerate(zip(past, new)):
        ids = table[s, p // P:-(-(p + n) // P)].long()
        assert torch.equal(cache.v_scale[ids], plain.v_scale[ids])
        last = ids[-1]
        assert torch.equal(cache.v[ids[:-1]], plain.v[ids[:-1]])
        live = (p + n - 1) % P + 1
        assert torch.equal(cache.v[last, ..., :live], plain.v[last, ..., :live])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("P,H,D,past,new,pad,kernel,size", [
    (16, 3, 64, [5], [40], 0, "read", 8192), (16, 3, 64, [5], [40], 1, "read_any", 8192),
    (64, 8, 128, [0, 9], [17000, 16500], 0, "read", 32768), (128, 5, 224, [1], [31000], 0, "read", 32768),
    (16, 3, 96, [7, 0, 3], [40000, 1, 76000], 0, "read", 8192), (32, 8, 128, [3], [33000], 3, "read_any", 32768)])
def test_read_forms(ops, dtype, P, H, D, past, new, pad, kernel, size):
    g = gen(P + H + D)
    cache, table = filled(g, P, H, D, past, new)
    n = sum(new)
    wide = torch.full((n, 2 * H * D + pad), 7.0, dtype=dtype, device="cuda")
    both = wide[:, pad:].unflatten(1, (2 * H, D))
    V.cache_read(ops, cache, batch_of(table, past, new), n, k=both[:, :H], v=both[:, H:])
    assert V.voc_dbg_last_kernel(ops) == (kernel, (size, P))
    at = torch.cat([torch.arange(p, p + m) for p, m in zip(past, new)]).cuda()
    b = torch.cat([torch.full((m,), s) for s, m in enumerate(new)]).cuda()
    for r in range(0, n, 8192):
        page, slot = table[b[r:r + 8192], at[r:r + 8192] // P].long(), at[r:r + 8192] % P
        want = (cache.k[page, :, slot].float() * cache.k_scale[page][..., None]).to(dtype)
        assert torch.equal(both[r:r + 8192, :H], want)
        want = (cache.v[page, :, :, slot].float() * cache.v_scale[page][..., None]).to(dtype)
        assert torch.equal(both[r:r + 8192, H:], want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim", [(9000, 32, 8, 64), (3000, 1, 0, 256), (70, 64, 16, 128), (20000, 3, 5, 32)])
def test_norm_rotate_of_many_tokens(ops, dtype, tokens, heads, kv_heads, dim):
    """Waves that share a token's heads, and waves that go on with further tokens."""
    g = gen(tokens)
    q, k = randn(g, tokens, heads, dim, dtype=dtype), randn(g, tokens, max(kv_heads, 1), dim, dtype=dtype)[:, :kv_heads]
    freq, w = frequencies(dim // 2), 1 + randn(g, dim, std=0.3)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    qo, ko = V.norm_rotate(ops, q, k, position=pos, freq=freq, q_weight=w, k_weight=w)
    check_turned(qo, q, w, freq, pos, False, 1e-6)
    check_turned(ko, k, w, freq, pos, False, 1e-6)


# ------------------------------------------------------- memory and streams
def calls_on(ops, n):
    """name -> (inputs, call(inputs, stream) -> new outputs), of sizes that
    nothing else in these tests has."""
    g = gen(121)
    cache, table = filled(g, 16, 8, 64, [30], [n])
    b, freq = batch_of(table, [30], [n]), frequencies(32)
    w, codes, s = torch.ones(64, device="cuda"), torch.ones(512, 512, dtype=torch.int8, device="cuda"), torch.ones(512, device="cuda")
    ads = V.Adapters(randn(g, 2, 16, 512, dtype=F16), randn(g, 2, 512, 16, dtype=F16))
    rows = lambda *shape, dtype=F32: torch.ones(n, *shape, device="cuda", dtype=dtype)     # noqa: E731
    return {
        "norm_rotate": (lambda: [rows(8, 64), rows(8, 64), rows(dtype=torch.int32)],
                        lambda x, t: V.norm_rotate(ops, x[0], x[1], position=x[2], freq=freq, q_weight=w, stream=t)),
        "norm_rotate_append": (lambda: [rows(8, 64), rows(8, 64), rows(8, 64)],
                               lambda x, t: [V.norm_rotate_append(ops, cache, b, *x, freq=freq, q_weight=w, stream=t)]),
        "cache_read": (lambda: [], lambda x, t: V.cache_read(ops, cache, b, n, dtype=F32, stream=t)),
        "matmul_int_adapters": (lambda: [rows(512, dtype=torch.int8), rows(), rows(dtype=torch.int32)],
                                lambda x, t: [V.matmul_int_adapters(ops, x[0], x[1], codes, s, ads, x[2], stream=t)]),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["norm_rotate", "norm_rotate_append", "cache_read", "matmul_int_adapters"])
def test_explicit_stream_keeps_memory(ops, name, raw):
    """While a call is pending on an explicit stream, the memory that it reads
    and writes is not handed out again on the current one, and its outputs are
    no memory that pending work of the current stream may still use."""
    n = 4111
    make, call = calls_on(ops, n)[name]
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    want = [x.clone() for x in call(make(), None)]
    torch.cuda.synchronize()
    sizes = [(x.shape, x.dtype) for x in make() + want]
    x = make()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    busy = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    taken = {t.data_ptr() for t in busy}
    del busy
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    y = call(x, stream)
    assert not taken & {t.data_ptr() for t in y}
    mine = {t.data_ptr() for t in x + list(y)}
    del x, y
    fresh = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(3)]
    pending = not s.query()
    assert not mine & {t.data_ptr() for t in fresh}
    assert pending
    x = make()
    s.wait_stream(torch.cuda.current_stream())
    y = call(x, stream)
    torch.cuda.current_stream().wait_stream(s)
    for got, right in zip(y, want):
        assert torch.equal(got, right)
    torch.cuda.synchronize()


def test_handles_at_once():
    """Two threads with a handle and a stream each, adapters and steps at once:
    the bits of one after the other (u lies in a handle's own workspace)."""
    g = gen(33)
    M, N, K = 700, 600, 512
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, device="cuda") * 0.02, torch.rand(N, device="cuda") * 0.001
    ads = V.Adapters(randn(g, 4, 32, K, dtype=F16, std=0.05), randn(g, 4, N, 32, dtype=F16))
    ids = [torch.randint(-1, 4, (M,), generator=g, device="cuda").to(torch.int32) for _ in range(2)]
    handles = [V.open_ops(0) for _ in range(2)]
    want = [V.matmul_int_adapters(handles[0], a, sa, b, sb, ads, i) for i in ids]
    torch.cuda.synchronize()
    bad = []

    def work(t):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                y = V.matmul_int_adapters(handles[t], a, sa, b, sb, ads, ids[t])
                if not torch.equal(y, want[t]):
                    bad.append(t)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for h in handles:
        V.voc_ops_destroy(h)
    assert not bad


def test_step_leaves_rows_between_sequences(ops):
    """Rows of the queries that belong to no sequence, before, between and
    behind, stay; so do the keys' and values' inputs."""
    g = gen(44)
    P, H, D = 16, 2, 64
    cache, table, q, k, v = cache_and_rows(g, P, H, D, 2, [0, 5], [30, 12], F16)
    rows = [torch.cat((x[:0], x.new_zeros(4, *x.shape[1:]), x, x.new_zeros(9, *x.shape[1:]))).contiguous() for x in (q, k, v)]
    b = V.KVBatch(table, i32([0, 5]), i32([4, 34, 46]), 30, 30)
    out = torch.full_like(rows[0], 3.0)
    V.norm_rotate_append(ops, cache, b, *rows, freq=frequencies(32), out=out)
    assert (out[:4] == 3).all() and (out[46:] == 3).all()
    want, _ = V.norm_rotate(ops, q, position=positions([0, 5], [30, 12]), freq=frequencies(32))
    assert torch.equal(out[4:46], want)
    k2, v2 = torch.full_like(rows[1], 3.0), torch.full_like(rows[2], 3.0)
    V.cache_read(ops, cache, b, 55, k=k2, v=v2)
    assert (k2[:4] == 3).all() and (k2[46:] == 3).all() and (v2[:4] == 3).all() and (v2[46:] == 3).all()
    assert (k2[4:46] != 3).any() and starts_of([30, 12])[-1] == 42
