"""The transformer stage with norms of query and key heads and with low-rank
adapters of the streams, against a plain 64-bit model, and its histories saved
and taken up again."""
import dataclasses
import math

import pytest
import torch

from dac_vocoder_decoding_amd import front as F
from dac_vocoder_decoding_amd import vocoder as V
from test_gpu_front import BOUND, biased

pytestmark = pytest.mark.gpu

SHAPE = F.Shape(channels=256, heads=8, kv_heads=4, head_dim=64, hidden=512, layers=2, window=9, qk_norm=True)
RANK = 5


def plain(shape, w, frames, voices, numbers):
    """The stage in 64 bits without quantisation (whole clip at once)."""
    w = {k: v.double() for k, v in w.items()}
    rows, c, t = frames.shape
    h = frames.double().transpose(1, 2)

    def norm(x, g):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g

    def rotate(x):
        half = torch.arange(0, shape.head_dim, 2, device=x.device, dtype=torch.float64)
        ang = torch.outer(torch.arange(t, device=x.device, dtype=torch.float64),
                          shape.rotary_base ** (-half / shape.head_dim))[None, :, None]
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()), -1).flatten(-2)

    def product(name, x):
        y = x @ w[name].t()
        for r, i in enumerate(numbers):
            if 0 <= i < len(voices) and name in voices[i]:
                down, up = (z.half().double() for z in voices[i][name])
                y[r] += x[r] @ down.t() @ up.t()
        return y

    i, j = torch.arange(t, device=h.device)[:, None], torch.arange(t, device=h.device)[None]
    hide = (j > i) | (j <= i - shape.window)
    for n in range(shape.layers):
        p = f"layers.{n}."
        qkv = product(p + "qkv", norm(h, w[p + "norm1"])).view(rows, t, -1, shape.head_dim)
        q, k = qkv[:, :, :shape.heads], qkv[:, :, shape.heads:shape.heads + shape.kv_heads]
        if shape.qk_norm:
            q, k = norm(q, w[p + "q_norm"]), norm(k, w[p + "k_norm"])
        q, k, v = rotate(q), rotate(k), qkv[:, :, shape.heads + shape.kv_heads:]
        g = shape.heads // shape.kv_heads
        q, k, v = (x.transpose(1, 2).contiguous() for x in (q, k.repeat_interleave(g, 2), v.repeat_interleave(g, 2)))
        z = (q @ k.transpose(2, 3).contiguous() / math.sqrt(shape.head_dim)).masked_fill(hide, -math.inf)
        a = (torch.softmax(z, -1) @ v).transpose(1, 2).reshape(rows, t, -1)
        h = h + product(p + "o", a)
        u = product(p + "up", norm(h, w[p + "norm2"])) + w[p + "up_bias"]
        h = h + product(p + "down", 0.5 * u * (1 + torch.erf(u / math.sqrt(2))))
    return norm(h, w["norm"]).transpose(1, 2)


def clip(seed, rows, t):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(rows, SHAPE.channels, t, generator=g, device="cuda")


def off(x, ref):
    return ((x.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("qk_norm", [True, False])
@pytest.mark.parametrize("steps", [[40], [1] * 12 + [28], [25, 15], [7, 1, 32]])
def test_front_with_adapters(qk_norm, steps):
    """Within the stage's roundings (the adapters' terms are not rounded to 8
    bits; two norms a layer add none), and a model with a planted mistake at
    least twice as far off."""
    shape = dataclasses.replace(SHAPE, qk_norm=qk_norm)
    w, frames, numbers = biased(shape, 5), clip(6, 4, 40), [1, -1, 0, 1]
    voices = [F.make_adapter(shape, RANK, 7), F.make_adapter(shape, RANK, 8)]
    del voices[0]["layers.1.o"]                            # a product without a term
    ref = plain(shape, w, frames, voices, numbers)
    mistakes = {"no adapters": plain(shape, w, frames, [], numbers), "other adapters": plain(shape, w, frames, voices[::-1], numbers)}
    if qk_norm:
        steep = {k: 3 * v if "q_norm" in k else v for k, v in w.items()}
        mistakes["no norm"] = plain(dataclasses.replace(shape, qk_norm=False), w, frames, voices, numbers)
        mistakes["three times the weights"] = plain(shape, steep, frames, voices, numbers)
    for name, x in mistakes.items():
        assert off(x, ref) > 2 * BOUND, (name, off(x, ref))
    front = F.Front(shape, w, rows=4, max_frames=40, adapters=2, rank=RANK)
    try:
        for i, v in enumerate(voices):
            front.set_adapter(i, v)
        ids = torch.tensor(numbers, device="cuda")
        out, at = [], 0
        for t in steps:
            out.append(front.step(frames[:, :, at:at + t].contiguous(), ids))
            at += t
        err = off(torch.cat(out, 2), ref)
        print(f"steps {steps[:3]}..: relative error {err:.4f}")
        assert err <= BOUND, err
    finally:
        torch.cuda.synchronize()
        front.close()


def test_front_without_options_is_what_it_was():
    """Streams without an adapter: the same bits as a Front without adapters."""
    shape = dataclasses.replace(SHAPE, qk_norm=False)
    w, frames = biased(shape, 9), clip(10, 3, 12)
    one, two = F.Front(shape, w, 3, 12), F.Front(shape, w, 3, 12, adapters=1, rank=4)
    try:
        two.set_adapter(0, F.make_adapter(shape, 4, 1))
        want = one.step(frames)
        assert torch.equal(two.step(frames), want)
        two.reset()
        assert torch.equal(two.step(frames, torch.full((3,), -1, device="cuda")), want)
    finally:
        torch.cuda.synchronize()
        one.close()
        two.close()


def test_front_saved_and_taken_up():
    """Another Front goes on from the saved histories: the same codes, scales to
    their roundings (a page's largest code is 127, so that its scale comes back
    as 127 s / 127), outputs within the stage's."""
    w, frames = biased(SHAPE, 3), clip(4, 3, 40)
    first, second = (F.Front(SHAPE, w, rows=3, max_frames=40) for _ in range(2))
    try:
        empty = first.save()
        out = [first.step(frames[:, :, :25].contiguous())]
        state = first.save()
        second.load(state)
        for a, b in zip(first.caches, second.caches):
            live = a.k_scale > 0
            assert torch.equal(live, b.k_scale > 0) and live.any()
            k = torch.arange(16, device="cuda")
            for c in range(2):                             # pages of 16, the second with 9 tokens
                ids = first.table[:, c].long()
                seen = k < (16 if c == 0 else 9)
                assert torch.equal(a.k[ids][:, :, seen], b.k[ids][:, :, seen]) and torch.equal(a.v[ids][..., seen], b.v[ids][..., seen])
            assert ((a.k_scale - b.k_scale).abs() <= 4 * 2.0 ** -24 * a.k_scale).all()
            assert ((a.v_scale - b.v_scale).abs() <= 4 * 2.0 ** -24 * a.v_scale).all()
        for n in (1, 14):
            x = frames[:, :, 25:26] if n == 1 else frames[:, :, 26:]
            out.append(second.step(x.contiguous()))
        assert off(torch.cat(out, 2), plain(SHAPE, w, frames, [], [-1] * 3)) <= BOUND
        second.load(empty)
        assert torch.equal(second.step(frames[:, :, :25].contiguous()), out[0])
        with pytest.raises(ValueError):
            second.load({"frames": 41, "layers": state["layers"]})
        with pytest.raises(ValueError):
            second.load({"frames": 25, "layers": state["layers"][:1]})
        with pytest.raises(ValueError):
            second.step(frames[:, :, :1].contiguous(), torch.zeros(3, device="cuda"))      # no adapters here
    finally:
        torch.cuda.synchronize()
        first.close()
        second.close()


def test_adapters_of_a_front_are_checked():
    front = F.Front(SHAPE, biased(SHAPE, 3), rows=2, max_frames=4, adapters=2, rank=4)
    try:
        with pytest.raises(ValueError):
            front.set_adapter(2, F.make_adapter(SHAPE, 4, 1))
        with pytest.raises(ValueError):
            front.set_adapter(0, F.make_adapter(SHAPE, 5, 1))
        with pytest.raises(ValueError):
            front.set_adapter(0, {"layers.2.o": (None, None)})
        with pytest.raises(ValueError):
            front.step(clip(1, 2, 1), torch.zeros(3, device="cuda"))
    finally:
        torch.cuda.synchronize()
        front.close()
