"""A transformer stage in 8 bits ahead of the causal stream decoder.

The codec that the causal decoder belongs to hands its frames through a small
transformer with a sliding window and a key/value cache first (qwentts.cpp
ARCHITECTURE page, "Audio tokenizer decoder", "Streaming decode (stateful
path)").  `Front` runs a transformer of that kind for many streams at once on
the library's 8-bit operators: weights and activations as rows of 8-bit codes,
the cache in 8-bit pages.  One step takes the next t frames of every stream and
returns the latent frames that vocoder_stream_decode takes.  It is a plain
decoder-only stack (RMS norms, rotary positions, a GELU widening): a codec's
own gates, layer scales and upsampler are not in it, and its output is the last
norm's 8-bit rows.

    front = Front(Shape(channels=1024, ...), make_weights(shape, seed), rows=32, max_frames=250)
    latent = front.step(frames)            # [rows, channels, t], t >= 1, any t per step
    pcm = vocoder.stream_decode(ctx, latent)

Per layer, with h the residual stream:

    q8 = rows8(norm(h + delta))            rms_norm (residual addition, norm, 8-bit rows)
    q, k, v = Wqkv q8                      matmul_int
    q, k rotated by their positions        (torch: elementwise)
    k, v -> cache; a = attention           cache_append, cache_attention
    delta = Wo rows8(a)                    quantize_rows, matmul_int
    q8 = rows8(norm(h + delta))            rms_norm
    delta = Wd rows8(gelu(Wu q8 + bu))     matmul_int with GELU, quantize_rows, matmul_int

`python -m dac_vocoder_decoding_amd.front` runs it ahead of the causal codec
workload (32 streams in 25-frame chunks) with random weights.
"""
from __future__ import annotations

import dataclasses

import torch

from . import vocoder as V


@dataclasses.dataclass(frozen=True)
class Shape:
    channels: int = 1024     # of the frames in and out
    heads: int = 16
    kv_heads: int = 16
    head_dim: int = 64
    hidden: int = 4096       # of the widening product
    layers: int = 2
    window: int = 72         # positions that a query sees, itself included (0: all)
    rotary_base: float = 10000.0


def make_weights(shape: Shape, seed: int, device="cuda") -> dict:
    """Random fp32 weights: products N(0, 1 / inputs), norms near 1, small biases."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*size, std):
        return torch.randn(*size, generator=g, device=device) * std

    c, qkv = shape.channels, (shape.heads + 2 * shape.kv_heads) * shape.head_dim
    out = {"norm": 1 + normal(c, std=0.1)}
    for i in range(shape.layers):
        p = f"layers.{i}."
        out[p + "norm1"], out[p + "norm2"] = 1 + normal(c, std=0.1), 1 + normal(c, std=0.1)
        out[p + "qkv"] = normal(qkv, c, std=c ** -0.5)
        out[p + "o"] = normal(c, shape.heads * shape.head_dim, std=(shape.heads * shape.head_dim) ** -0.5)
        out[p + "up"], out[p + "up_bias"] = normal(shape.hidden, c, std=c ** -0.5), normal(shape.hidden, std=0.01)
        out[p + "down"] = normal(c, shape.hidden, std=shape.hidden ** -0.5)
    return out


class Front:
    """The stage's 8-bit weights and the caches of `rows` streams of up to
    max_frames frames."""

    def __init__(self, shape: Shape, weights: dict, rows: int, max_frames: int, page_tokens: int = 16,
                 device: int = 0):
        self.shape, self.rows, self.max_frames = shape, rows, max_frames
        self.ops = V.open_ops(device)
        self.device = torch.device("cuda", device)
        self.w = {}
        for name, w in weights.items():
            w = w.to(self.device, torch.float32).contiguous()
            self.w[name] = V.quantize_rows(self.ops, w) if w.dim() == 2 else w
        per = -(-max_frames // page_tokens)
        self.caches = [V.KVCache(rows * per, page_tokens, shape.kv_heads, shape.head_dim, self.device)
                       for _ in range(shape.layers)]
        self.table = torch.arange(rows * per, dtype=torch.int32, device=self.device).view(rows, per)
        self.past = torch.zeros(rows, dtype=torch.int32, device=self.device)
        self.frames = 0                                   # frames that every stream has received
        half = torch.arange(0, shape.head_dim, 2, device=self.device, dtype=torch.float32)
        angle = torch.outer(torch.arange(max_frames, device=self.device), shape.rotary_base ** (-half / shape.head_dim))
        self.cos, self.sin = angle.cos().half(), angle.sin().half()

    def close(self) -> None:
        """Releases the operators' handle (after the streams were synchronized)."""
        if self.ops is not None:
            V.voc_ops_destroy(self.ops)
            self.ops = None

    def reset(self) -> None:
        """Starts every stream with an empty history."""
        self.frames = 0
        self.past.zero_()

    def _rotate(self, x, t: int) -> None:
        """Rotates x [rows * t, heads, head_dim] by its positions, in place."""
        c = self.cos[self.frames:self.frames + t].repeat(self.rows, 1)[:, None]
        s = self.sin[self.frames:self.frames + t].repeat(self.rows, 1)[:, None]
        a, b = x[..., 0::2], x[..., 1::2]
        a_new, b_new = a * c - b * s, b * c + a * s
        x[..., 0::2], x[..., 1::2] = a_new, b_new

    def step(self, frames):
        """Latent frames [rows, channels, t] (fp32) of the next t frames
        [rows, channels, t] (fp32) of every stream."""
        sh, ops = self.shape, self.ops
        rows, c, t = frames.shape
        if (rows, c) != (self.rows, sh.channels) or t < 1 or self.frames + t > self.max_frames:
            raise ValueError(f"frames {tuple(frames.shape)}: [{self.rows}, {sh.channels}, t] is needed, and "
                             f"{self.max_frames - self.frames} more frames fit the cache")
        starts = torch.arange(0, rows * t + 1, t, dtype=torch.int32, device=self.device)
        batch = V.KVBatch(self.table, self.past, starts, t, self.frames + t)
        h, delta = frames.transpose(1, 2).reshape(rows * t, c).half(), None
        nq, nk, d = sh.heads, sh.kv_heads, sh.head_dim
        for i in range(sh.layers):
            w = lambda name: self.w[f"layers.{i}.{name}"]          # noqa: E731
            q8, s, h = V.rms_norm(ops, h, w("norm1"), residual=delta)
            qkv = V.matmul_int(ops, q8, s, *w("qkv"), dtype=torch.float16).view(rows * t, nq + 2 * nk, d)
            self._rotate(qkv[:, :nq + nk], t)
            V.cache_append(ops, self.caches[i], batch, qkv[:, nq:nq + nk], qkv[:, nq + nk:])
            a = V.cache_attention(ops, self.caches[i], batch, qkv[:, :nq], window=sh.window)
            delta = V.matmul_int(ops, *V.quantize_rows(ops, a.view(rows * t, nq * d)), *w("o"), dtype=torch.float16)
            q8, s, h = V.rms_norm(ops, h, w("norm2"), residual=delta)
            u = V.matmul_int(ops, q8, s, *w("up"), bias=w("up_bias"), gelu=True, dtype=torch.float16)
            delta = V.matmul_int(ops, *V.quantize_rows(ops, u), *w("down"), dtype=torch.float16)
        q8, s, _ = V.rms_norm(ops, h, self.w["norm"], residual=delta)
        self.frames += t
        self.past += t
        out = torch.mul(q8, s[:, None])                   # the normalised rows, as the decoder's latent
        return out.view(rows, t, c).transpose(1, 2).contiguous()


def main() -> int:
    import time

    from . import inputs as I
    cfg = I.config(7)
    rows, ck, total = cfg["batch"], cfg["chunk"], cfg["frames"]
    shape = Shape(channels=cfg["latent_channels"])
    front = Front(shape, make_weights(shape, cfg["seed"]), rows, total)
    ctx = V.open_context(cfg, I.make_weights(cfg))
    frames = torch.from_numpy(I.make_latent(cfg)).cuda()
    try:
        for timed in (False, True):
            front.reset()
            V.check(V.vocoder_stream_reset(ctx, rows), ctx)
            torch.cuda.synchronize()
            t_front = t_all = 0.0
            for k in range(0, total, ck):
                t0 = time.perf_counter()
                latent = front.step(frames[:, :, k:k + ck].contiguous())
                torch.cuda.synchronize()
                t1 = time.perf_counter()
                V.stream_decode(ctx, latent)
                torch.cuda.synchronize()
                t_front, t_all = t_front + t1 - t0, t_all + time.perf_counter() - t0
            if timed:
                n = total // ck
                print(f"{rows} streams, {n} chunks of {ck} frames: transformer stage {1e3 * t_front / n:.3f} ms a chunk, "
                      f"with the decoder {1e3 * t_all / n:.3f} ms "
                      f"({I.audio_seconds(cfg, rows, total) / t_all:.0f} audio-s/s)")
    finally:
        torch.cuda.synchronize()
        V.vocoder_destroy(ctx)
        front.close()
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
