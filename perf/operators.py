"""What is measured of the 8-bit transformer operators: the cases, their plain forms in 32 bits, and their
definitions in 64 bits.

The operators are the ones a codec's transformer stage runs ahead of the causal decoder: the RMS norm with residual
addition and 8-bit rows, the 8-bit integer product, the 8-bit paged cache's append and the attention over it.
Stream and frame counts (32 streams, 25-frame chunks, 250 and 5168 frames, windows of 689, 1024 channels, 1536 wide
convs) are those of the decoder's own workloads; head counts and cache lengths are generic.

A case's sizes, the ragged ones among them, follow from the case alone; its values follow from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -100          # a block whose largest magnitude is below this is held as zeros
INV127 = torch.tensor(1.0 / 127.0, dtype=torch.float32).item()


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One frame of 32 streams ahead of a layer: the smallest call, all latency.
        dict(name="norm_frame_f16", op="norm", rows=32, width=1024, dtype="f16", residual=True),
        # A song's 14 windows of 689 frames, both sides, 4096 wide: one pass over memory.
        dict(name="norm_song_bf16", op="norm", rows=19292, width=4096, dtype="bf16", residual=True),
        # Activations in 32 bits of an odd width, quantised in front of a product.
        dict(name="quantize_odd_f32", op="quantize", rows=1378, width=1501, dtype="f32", residual=False),
        # One frame of 32 streams through the widening product (1024 -> 4096, GELU): reads the weights once.
        dict(name="product_frame_f16", op="product", m=32, n=4096, k=1024, dtype="f16", bias=True, gelu=True, pad=0),
        # Odd sizes and rows that start at odd addresses.
        dict(name="product_odd_f32", op="product", m=689, n=1000, k=1501, dtype="f32", bias=True, gelu=False, pad=6),
        # 32 streams of 250 frames in one call, the largest product: bound by the matrix cores.
        dict(name="product_clip_bf16", op="product", m=8000, n=8192, k=4096, dtype="bf16", bias=False, gelu=False, pad=0),
        # The new frame of 32 streams into their last pages.
        dict(name="append_frame_f16", op="append", batch=32, new=1, past=100, kv_heads=8, dim=128, page=64,
             dtype="f16", ragged=3),
        # 8 prompts of up to 5168 frames into an empty cache, pages that end inside the prompt.
        dict(name="append_prompt_bf16", op="append", batch=8, new=5168, past=0, kv_heads=8, dim=128, page=32,
             dtype="bf16", ragged=5),
        # One frame of 32 streams of 16 heads over the last 250 frames.
        dict(name="attend_frame_f16", op="attend", batch=32, new=1, past=250, heads=16, kv_heads=16, dim=64, page=32,
             dtype="f16", causal=True, window=0, ragged=7),
        # One token of 4 streams over a very long cache, four query heads to a cache head: bound by the cache's bytes.
        dict(name="attend_long_bf16", op="attend", batch=4, new=1, past=65536, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", causal=True, window=0, ragged=9),
        # A 25-frame chunk of 32 streams with a sliding window.
        dict(name="attend_chunk_bf16", op="attend", batch=32, new=25, past=689, heads=16, kv_heads=16, dim=64, page=16,
             dtype="bf16", causal=True, window=72, ragged=11),
        # 2 prompts of up to 5168 frames, causal: bound by the matrix cores.
        dict(name="attend_prompt_bf16", op="attend", batch=2, new=5168, past=0, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", causal=True, window=0, ragged=13),
    ]


def draw(rng):
    def log(lo, hi, of=1):
        n = of * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if n != 3 * 1024 else n + of

    op = rng.choice(("norm", "quantize", "product", "product", "append", "attend", "attend", "attend"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op in ("norm", "quantize"):
        width = rng.choice((log(64, 8192), log(8, 1024, 8)))
        rows = min(log(1, 20000), 70000000 // width)
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=op == "norm" and rng.random() < 0.7)
    if op == "product":
        n, k = rng.choice((log(16, 8192), log(1, 128, 64))), rng.choice((log(16, 4096), log(1, 64, 64)))
        return dict(op=op, m=rng.choice((log(1, 64), log(1, 8000))), n=n, k=k, dtype=dtype, bias=rng.random() < 0.5,
                    gelu=rng.random() < 0.3, pad=rng.choice((0, 0, 16, 5)))
    page, dim = rng.choice((16, 32, 64, 128)), rng.choice((32, 64, 96, 128, 192, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    if op == "append":
        new = rng.choice((1, log(1, 64), log(64, 5168)))
        batch = max(1, min(log(1, 32), 5000000 // (new * kv_heads * dim)))
        return dict(op=op, batch=batch, new=new, past=rng.choice((0, log(1, 1000))), kv_heads=kv_heads, dim=dim,
                    page=page, dtype=dtype, ragged=rng.randrange(1, 1 << 20))
    heads = kv_heads * rng.choice((1, 1, 2, 4, 5))
    form = rng.choice(("single", "single", "chunk", "prompt"))
    if form == "single":
        past, new = log(1, 65536), 1
        batch = max(1, min(log(1, 32), 16000000 // (past * kv_heads * dim)))
    elif form == "chunk":
        past, new = log(1, 4096), log(2, 64)
        batch = max(1, min(log(1, 32), 16000000 // (past * kv_heads * dim)))
    else:
        past, new = rng.choice((0, log(1, 1000))), log(64, 2600)
        batch = max(1, min(4, 500000000 // (new * (new + past) * heads)))
    return dict(op=op, batch=batch, new=new, past=past, heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype,
                causal=rng.random() < 0.8, window=rng.choice((0, 0, log(1, 1000))), ragged=rng.randrange(1, 1 << 20))


def lengths(case):
    """Tokens held before and new tokens of each sequence: the first has the case's own numbers, the others up to
    40 % less (a single new token stays one)."""
    r = random.Random(case["ragged"])
    past, new = [case["past"]], [case["new"]]
    for _ in range(case["batch"] - 1):
        past.append(int(case["past"] * r.uniform(0.6, 1.0)))
        new.append(max(1, int(case["new"] * r.uniform(0.6, 1.0))))
    return past, new


def visible_pairs(case):
    """Visible (query, key) pairs of one head, and tokens that some query sees, over all sequences."""
    pairs = tokens = 0
    for past, new in zip(*lengths(case)):
        w = case["window"] or past + new
        first = past + new
        for i in range(new):
            last = past + i if case["causal"] else past + new - 1
            lo = max(0, past + i - w + 1)
            pairs += max(0, last - lo + 1)
            first = min(first, lo)
        tokens += past + new - first
    return pairs, tokens


def work(case):
    op, e = case["op"], torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if op in ("norm", "quantize"):
        n = case["rows"] * case["width"]
        reads = e * n * (2 if case["residual"] else 1)
        return {"bytes": reads + (e * n if op == "norm" else 0) + n + 4 * case["rows"], "flops": 8 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + e * m * n + 4 * (m + n), "flops": 2 * m * n * k}
    past, new = lengths(case)
    if op == "append":
        n = sum(new) * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * (e + 1), "flops": 6 * n}
    pairs, tokens = visible_pairs(case)
    rows = sum(new) * case["heads"] * case["dim"]
    return {"bytes": 2 * e * rows + 2 * tokens * case["kv_heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ----------------------------------------------------------------- inputs
_handle = None


def _ops():
    """The operators' handle, opened once as a program does."""
    global _handle
    from dac_vocoder_decoding_amd import vocoder as V
    if _handle is None:
        _handle = V.open_ops(0)
    return V, _handle


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.float32, spread=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * spread).to(dtype)


def _codes(g, rows, cols, pad):
    """Signed 8-bit rows as a quantiser leaves them (about a quarter of the range in standard deviation), in rows of
    cols + pad bytes."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    return x[:, :cols]


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]
    s = dict(op=op, case=case, dt=dt)
    if op in ("norm", "quantize"):
        rows, width = case["rows"], case["width"]
        # A residual stream: a few channels are much larger than the rest.
        gain = torch.exp(_normal(g, width, spread=0.7))
        s["x"] = (_normal(g, rows, width) * gain).to(dt)
        if case["residual"]:
            s["r"] = (_normal(g, rows, width, spread=4.0) * gain).to(dt)
        s["w"] = 1.0 + _normal(g, width, spread=0.2)
        s["values"] = torch.empty(rows, width, dtype=torch.float16, device="cuda")
    elif op == "product":
        s["a"], s["b"] = _codes(g, case["m"], case["k"], case["pad"]), _codes(g, case["n"], case["k"], case["pad"])
        s["sa"] = torch.rand(case["m"], generator=g, device="cuda") * 0.03 + 0.01
        s["sb"] = (torch.rand(case["n"], generator=g, device="cuda") * 0.03 + 0.01) / math.sqrt(case["k"])
        s["bias"] = _normal(g, case["n"], spread=0.1) if case["bias"] else None
    else:
        past, new = lengths(case)
        H, D, P = case["kv_heads"], case["dim"], case["page"]
        per = max(-(-(p + n) // P) for p, n in zip(past, new)) + 1
        pages = per * case["batch"]
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(case["batch"], per)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s.update(past=torch.tensor(past, dtype=torch.int32, device="cuda"), table=table, max_new=max(new),
                 max_total=max(p + n for p, n in zip(past, new)), tokens=starts[-1],
                 starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        held = past if op == "append" else [p + n for p, n in zip(past, new)]
        # Pages that hold tokens: a key page [token][dim] and a value page [dim][token], one scale a page and head.
        pos = torch.arange(per * P, device="cuda").reshape(1, per, P)
        live = torch.zeros(pages, P, dtype=torch.bool, device="cuda")
        live[table.long()] = pos < torch.tensor(held, device="cuda").reshape(-1, 1, 1)
        k = torch.randn(pages, H, P, D, generator=g, device="cuda", dtype=torch.float16).mul_(36).round_().clamp_(-127, 127)
        v = torch.randn(pages, H, D, P, generator=g, device="cuda", dtype=torch.float16).mul_(36).round_().clamp_(-127, 127)
        s["k"] = (k * live[:, None, :, None]).to(torch.int8)
        s["v"] = (v * live[:, None, None, :]).to(torch.int8)
        some = live.any(1)[:, None].float()
        s["ks"] = (torch.rand(pages, H, generator=g, device="cuda") * 0.012 + 0.020) * some
        s["vs"] = (torch.rand(pages, H, generator=g, device="cuda") * 0.012 + 0.020) * some
        if op == "append":
            # Keys and values are slices of the rows that one product wrote.
            both = _normal(g, s["tokens"], 2 * H, D, dtype=dt)
            s["new_k"], s["new_v"] = both[:, :H], both[:, H:]
            s["k_values"] = torch.empty(s["k"].shape, dtype=torch.float16, device="cuda")
            s["v_values"] = torch.empty(s["v"].shape, dtype=torch.float16, device="cuda")
        else:
            s["q"] = _normal(g, s["tokens"], case["heads"], D, dtype=dt)
    if own:
        V, s["ops"] = _ops()
        s["V"] = V
        if op in ("append", "attend"):
            s["cache"] = V.KVCache.from_tensors(s["k"], s["v"], s["ks"], s["vs"])
            s["batch"] = V.KVBatch(s["table"], s["past"], s["starts"], s["max_new"], s["max_total"])
    return s


# -------------------------------------------------------------- plain forms
def _scale_of(amax):
    return torch.where(amax < TINY, torch.zeros_like(amax), amax * INV127)


def _inverse(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def _plain_norm(s):
    x = s["x"].float()
    h = None
    if s["op"] == "norm":
        h = s["x"]
        if "r" in s:
            h = (x + s["r"].float()).to(s["dt"])
        x = h.float()
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * s["w"]
    scale = _scale_of(x.abs().amax(1))
    codes = (x * _inverse(scale)[:, None]).round().clamp(-127, 127)
    values = (codes * scale[:, None]).to(torch.float16)
    return (values, scale) if h is None else (values, scale, h)


def _plain_product(s):
    y = (s["a"].float() @ s["b"].float().t()) * s["sa"][:, None] * s["sb"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"]["gelu"]:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y.to(s["dt"])


def _plain_append(s):
    c = s["case"]
    P, past = c["page"], s["past"].long()
    touched = (s["max_new"] + P - 1) // P + 1
    column = past[:, None] // P + torch.arange(touched, device="cuda")
    page = torch.gather(s["table"].long(), 1, column.clamp(max=s["table"].shape[1] - 1))
    pos = (column[:, :, None] * P + torch.arange(P, device="cuda"))           # [B, touched, P]
    index = pos - past[:, None, None]
    count = (s["starts"][1:] - s["starts"][:-1]).long()[:, None, None]
    fresh, old = (index >= 0) & (index < count), index < 0
    token = (s["starts"][:-1].long()[:, None, None] + index).clamp(0, s["tokens"] - 1)
    write = fresh.any(2) & (column < s["table"].shape[1])
    # Pages past a sequence's last are written back as they are, each to a place of its own.
    spare = s["k"].shape[0]
    out = []
    for new, codes, scale, swap in ((s["new_k"], s["k"], s["ks"], False), (s["new_v"], s["v"], s["vs"], True)):
        x = torch.where(fresh[..., None, None], new.float()[token], torch.zeros((), device="cuda"))
        x = x.transpose(2, 3)                                                  # [B, touched, H, P, D]
        before = torch.where(old.any(2)[..., None], scale[page], torch.zeros((), device="cuda"))
        after = torch.maximum(before, _scale_of(x.abs().amax((3, 4))))
        ratio = (before * _inverse(after))[..., None, None]
        was = codes[page].float()
        was = was.transpose(3, 4) if swap else was
        kept = torch.where(old[:, :, None, :, None], (was * ratio).round(), was)
        coded = torch.where(fresh[:, :, None, :, None], (x * _inverse(after)[..., None, None]).round().clamp(-127, 127), kept)
        coded = (coded.transpose(3, 4) if swap else coded).to(torch.int8)
        where = torch.where(write, page, spare + torch.arange(page.numel(), device="cuda").reshape(page.shape))
        grown = torch.cat((codes, codes.new_empty(page.numel(), *codes.shape[1:])))
        grown[where] = coded
        codes.copy_(grown[:spare])
        grown = torch.cat((scale, scale.new_empty(page.numel(), scale.shape[1])))
        grown[where] = after
        scale.copy_(grown[:spare])
        out.append((codes.float() * scale[:, :, None, None]).to(torch.float16))
    return out[0], out[1], s["ks"], s["vs"]


def _plain_attend(s):
    c = s["case"]
    P, D, H = c["page"], c["dim"], c["kv_heads"]
    g = c["heads"] // H
    used = -(-s["max_total"] // P)
    page = s["table"][:, :used].long()
    B, L = page.shape[0], used * P
    k = s["k"][page].float() * s["ks"][page][..., None, None]                  # [B, pages, H, P, D]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    v = s["v"][page].float() * s["vs"][page][..., None, None]                  # [B, pages, H, D, P]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, L, D)
    n = s["max_new"]
    i = torch.arange(n, device="cuda")
    token = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[token].reshape(B, n, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * n, D)
    score = (q @ k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(D)).reshape(B, H, g, n, L)
    at = s["past"].long()[:, None] + i                                         # [B, n]
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    j = torch.arange(L, device="cuda")
    seen = (j < (s["past"].long() + count)[:, None, None]).expand(B, n, L)
    if c["causal"]:
        seen = seen & (j <= at[..., None])
    if c["window"]:
        seen = seen & (j > at[..., None] - c["window"])
    seen = seen[:, None, None]
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, g * n, L) @ v).reshape(B, H, g, n, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), t, right=True)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, c["heads"], D)[b, t - s["starts"].long()[b]].to(s["dt"])


PLAIN = {"norm": _plain_norm, "quantize": _plain_norm, "product": _plain_product, "append": _plain_append,
         "attend": _plain_attend}


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    V, ops, c = s["V"], s["ops"], s["case"]
    if s["op"] == "norm":
        codes, scale, h = V.rms_norm(ops, s["x"], s["w"], eps=1e-6, residual=s.get("r"))
        return torch.mul(codes, scale[:, None], out=s["values"]), scale, h
    if s["op"] == "quantize":
        codes, scale = V.quantize_rows(ops, s["x"])
        return torch.mul(codes, scale[:, None], out=s["values"]), scale
    if s["op"] == "product":
        return V.matmul_int(ops, s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], gelu=c["gelu"], dtype=s["dt"])
    if s["op"] == "append":
        V.cache_append(ops, s["cache"], s["batch"], s["new_k"], s["new_v"])
        return (torch.mul(s["k"], s["ks"][:, :, None, None], out=s["k_values"]),
                torch.mul(s["v"], s["vs"][:, :, None, None], out=s["v_values"]), s["ks"], s["vs"])
    return V.cache_attention(ops, s["cache"], s["batch"], s["q"], causal=c["causal"], window=c["window"])


# -------------------------------------------------- the definitions, 64 bits
def _rows_exact(y):
    amax = y.abs().max(1).values
    scale = torch.where(amax < TINY, 0.0, amax / 127)
    codes = torch.where(scale[:, None] > 0, torch.round(y / scale[:, None]), 0.0)
    return codes * scale[:, None], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _rows_exact(s["x"].double())
    if op == "norm":
        h = s["x"].double() + (s["r"].double() if "r" in s else 0.0)
        kept = h.to(s["dt"]).double()
        y = kept / torch.sqrt(kept.square().sum(1, keepdim=True) / case["width"] + 1e-6) * s["w"].double()
        return (*_rows_exact(y), h)
    if op == "product":
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for r in range(0, case["m"], 2000):
            y[r:r + 2000] = s["a"][r:r + 2000].double().matmul(s["b"].double().t())
        y *= s["sa"].double()[:, None] * s["sb"].double()[None]
        y += s["bias"].double() if case["bias"] else 0.0
        return torch.special.ndtr(y) * y if case["gelu"] else y
    past, new = lengths(case)
    P, H = case["page"], case["kv_heads"]
    table = s["table"].tolist()
    if op == "append":
        k, v = s["k"].double(), s["v"].double().transpose(2, 3).contiguous()
        ks, vs = s["ks"].double(), s["vs"].double()
        base = 0
        for b in range(case["batch"]):
            for t0 in range(past[b] // P * P, past[b] + new[b], P):
                page, lo, hi = table[b][t0 // P], max(t0, past[b]), min(t0 + P, past[b] + new[b])
                rows = slice(base + lo - past[b], base + hi - past[b])
                for codes, scale, x in ((k, ks, s["new_k"]), (v, vs, s["new_v"])):
                    x = x[rows].double().transpose(0, 1)                       # [H, tokens, D]
                    amax = x.abs().reshape(H, -1).max(1).values
                    was = scale[page] if lo > t0 else torch.zeros_like(amax)
                    now = torch.maximum(was, torch.where(amax < TINY, 0.0, amax / 127))
                    safe = torch.where(now > 0, now, 1.0)[:, None, None]
                    if lo > t0:
                        codes[page][:, :lo - t0] = torch.round(codes[page][:, :lo - t0] * was[:, None, None] / safe)
                    codes[page][:, lo - t0:hi - t0] = torch.round(x / safe)
                    scale[page] = now
            base += new[b]
        return k * ks[:, :, None, None], (v * vs[:, :, None, None]).transpose(2, 3), ks, vs
    D, g, base = case["dim"], case["heads"] // H, 0
    out = torch.zeros(s["tokens"], case["heads"], D, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        total = past[b] + new[b]
        ids = torch.tensor(table[b][:-(-total // P)], device="cuda")
        at = torch.arange(past[b], total, device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        hide = (j > at) if case["causal"] else (j < 0)
        if case["window"]:
            hide = hide | (at - j >= case["window"])
        for h in range(H):
            k = (s["k"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).reshape(-1, D)[:total]
            v = (s["v"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:total]
            for m in range(h * g, h * g + g):
                z = s["q"][base:base + new[b], m].double() @ k.t() / math.sqrt(D)
                out[base:base + new[b], m] = torch.softmax(z.masked_fill(hide, -math.inf), 1) @ v
        base += new[b]
    return out
